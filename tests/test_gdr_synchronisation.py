"""The order of shared-memory accesses and barriers in the gated-delta-rule kernels, on the CPU.

Whether two warps can meet in a buffer, or miss each other at a barrier, does not show in a run that
happens to be timed well.  These tests take the accesses, barriers and waits as they stand in the
sources and go through every order that the barriers allow."""
import os
import re

from kda_delta_rule_chunkwise_b200 import build as kbuild


def source(name):
    with open(os.path.join(kbuild.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block_behind(text, start):
    """The braces' content that follows `start`."""
    at = text.index("{", text.index(start))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError(start)


def test_no_buffer_of_the_decode_kernel_is_read_and_written_between_two_barriers():
    """Between two barriers any warp may be ahead of any other: a buffer half that one statement writes
    there is touched by no other statement."""
    text = source("gdr_token.cu")
    published = sorted(set(re.findall(r"(\w+)\[b\]", block_behind(text, "auto publish = [&](int b)"))))
    assert published == ["gb", "ks", "qs", "vs"]
    body = block_behind(text, "for (int t = 0; t < len; ++t)")
    shared = published + ["red_p", "red_y", "dl", "kq"]
    events = []   # of one token: "barrier", or (buffer, offset of its half, written?)
    pattern = r"__syncthreads\(\)|publish\(b \^ 1\)|\b(%s)\[b\]((?:\[[^\]]*\])*)(\s*=[^=])?" % "|".join(shared)
    for m in re.finditer(pattern, body):
        if m.group(0).startswith("__sync"):
            events.append("barrier")
        elif m.group(0).startswith("publish"):
            events += [(name, 1, True) for name in published]
        else:
            events.append((m.group(1), 0, m.group(3) is not None))
    assert events.count("barrier") == 2 and ("ks", 1, True) in events and ("dl", 0, True) in events
    interval, seen = 0, {}
    for t in range(6):
        for e in events:
            if e == "barrier":
                interval += 1
                continue
            name, ahead, written = e
            others = seen.setdefault((interval, name, (t + ahead) & 1), set())
            others.add((t + ahead, written))
            assert not (any(w for _, w in others) and len(others) > 1), \
                f"{name}[{(t + ahead) & 1}] is written and used by tokens {sorted(others)} without a barrier between"
