"""The order of shared-memory accesses and barriers in the gated-delta-rule and block-norm kernels, on the CPU.

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


def test_two_warps_of_a_column_group_never_miss_each_other():
    """Each warp hands its half sums over, arrives at a barrier and waits at one, chunk after chunk.  A wait
    asks for a parity, so a warp that is late by two phases would wait for ever: no order of
    the two warps' steps may come to a halt, or let a warp read a buffer too early or too late."""
    pipe = source("gdr_common.cuh")
    groups = 2
    number, arrivals = re.search(r"i < (.*); \+\+i\) mbar_init\(swapped \+ i, (.*)\);", pipe).groups()
    assert f"(2 * ST + {number} + OW * ST) * 8" in pipe and f"handed = swapped + {number};" in pipe   # their place
    number, arrivals = (eval(e, {"NCW": groups, "KS": 2}) for e in (number, arrivals))
    for name, step in (("gdr_chunk.cu", "ci"), ("gdr_backward.cu", "it")):
        text = source(name)
        (arrive,) = re.findall(r"mbar_arrive\(pipe\.swapped \+ (.*)\);", text)
        (index, parity), = re.findall(r"pipe\.wait\(pipe\.swapped \+ (.*), ([^,\n]*)\);\n", text)
        chunks = 7

        def value(expr, part, chunk, group=0):
            return eval(expr, {"group": group, "part": part, step: chunk})   # C and Python agree on these operators

        used = [{value(e, part, c, g) for e in (arrive, index) for part in range(2) for c in range(chunks)}
                for g in range(groups)]
        assert not used[0] & used[1] and all(0 <= i < number for u in used for i in u)
        # a warp's steps: 4 c write its half of buffer c & 1; 4 c + 1 arrive; 4 c + 2 wait; 4 c + 3 read the other's
        todo, known = [((0, 0), (0,) * number)], set()
        while todo:
            state = todo.pop()
            if state in known:
                continue
            known.add(state)
            at, arrived = state
            moved = False
            for part in range(2):
                c, what = divmod(at[part], 4)
                if c == chunks:
                    continue
                after = list(arrived)
                if what == 1:
                    after[value(arrive, part, c)] += 1
                elif what == 2 and arrived[value(index, part, c)] // arrivals & 1 == value(parity, part, c):
                    continue   # the phase asked for is the one in progress
                elif what == 3:
                    other = at[part ^ 1]
                    assert 4 * c + 1 < other <= 4 * (c + 2), (name, "read at the wrong time", at)
                moved = True
                todo.append((tuple(a + (i == part) for i, a in enumerate(at)), tuple(after)))
            assert moved or at == (4 * chunks, 4 * chunks), (name, "both warps wait", at, arrived)


def test_no_wait_that_gives_up_leaves_copies_behind():
    """A kernel that copies into its shared memory waits for those copies before it leaves early."""
    for name in ("gdr_common.cuh", "gdr_backward.cu", "block_norm.cu"):
        assert not re.search(r"wait\w*\([^;{}]*\)\)?\s*return;", source(name)), name
    load = block_behind(source("gdr_common.cuh"), "__device__ __forceinline__ void load(")
    assert "mbar_wait(full + c % ST, (c / ST) & 1, err)" in load.rsplit("__syncwarp", 1)[1]
    grads = block_behind(source("gdr_backward.cu"), "gdr_grads_kernel(GradsArgs a)")
    assert "mbar_wait(bar, parity ^ 1u, a.err)" in block_behind(grads, "if (__syncthreads_or(late))")
    for kernel in ("block_norm_kernel(BlockNormArgs a)", "block_norm_backward_kernel(BlockNormArgs a)"):
        body = block_behind(source("block_norm.cu"), kernel)
        assert "Rows::drain(a, base, step, stage, parity, bars)" in block_behind(body, "if (abort)")
