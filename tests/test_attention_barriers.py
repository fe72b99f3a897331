"""The tile kernel's start without a GPU: its load warp arrives at the first barrier and goes on,
so every order of the warps is walked through a model of the hardware's barriers (they count
arrivals, whoever makes them), with the barrier numbers that the source gives."""
import os
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "q8_int8_block_gb300", "csrc", "q8_attn.cu")
END = 0  # __syncthreads


def _number(text, instruction):
    """The barrier that the kernel's only `instruction` over all its threads names."""
    found = re.findall(r'asm volatile\("%s (%%?\w+), [^;]*;" ::([^:]*kTileThreads[^:]*):' % re.escape(instruction), text)
    assert len(found) == 1, (instruction, found)
    where, operands = found[0]
    if not where.startswith("%"):
        return int(where)
    name = re.findall(r'"n"\((\w+)\)', operands)[int(where[1:])]
    return int(re.search(r"constexpr int %s = (\d+);" % name, text)[1])


def _walk(arrive, sync, warps):
    """All orders of a load warp, which arrives and then meets the others at the end, and warps
    that wait at the start: returns what can go wrong."""
    programs = [[("arrive", arrive), ("sync", END)]] + [[("sync", sync), ("sync", END)]] * (warps - 1)
    start = (tuple([0] * warps), tuple([False] * warps), ())  # places, waiting, arrivals of each barrier
    todo, seen, wrong = [start], {start}, set()
    while todo:
        at, waiting, counts = todo.pop()
        moves = [w for w in range(warps) if not waiting[w] and at[w] < 2]
        if not moves and any(waiting):
            wrong.add("stuck")
        for w in moves:
            kind, bar = programs[w][at[w]]
            n, a, wt = dict(counts), list(at), list(waiting)
            n[bar] = n.get(bar, 0) + 1
            if kind == "sync":
                wt[w] = True
            else:
                a[w] += 1
            if n[bar] == warps:  # all that wait there go on
                n[bar] = 0
                for x in range(warps):
                    if wt[x] and programs[x][a[x]] == ("sync", bar):
                        # past the start while a warp has not come to it
                        if a[x] == 0 and any(a[y] == 0 and not wt[y] for y in range(warps)):
                            wrong.add("early")
                for x in range(warps):
                    if wt[x] and programs[x][a[x]] == ("sync", bar):
                        wt[x], a[x] = False, a[x] + 1
            state = (tuple(a), tuple(wt), tuple(sorted(n.items())))
            if state not in seen:
                seen.add(state)
                todo.append(state)
    return wrong


def test_the_model_tells_a_shared_number_from_one_of_its_own():
    assert _walk(0, 0, 4) == {"early", "stuck"} and _walk(11, 11, 4) == set()
    assert "stuck" in _walk(11, 12, 4)


def test_no_warp_starts_before_the_others_have_come():
    with open(SRC) as f:
        text = f.read()
    arrive, sync = _number(text, "bar.arrive"), _number(text, "bar.sync")
    assert _walk(arrive, sync, 5) == set()
    assert arrive not in range(0, 11)  # nor is it one of the softmax warps' barriers
