"""The barriers between a prompt tile's MMA issuer and its softmax warps, as a
model walked through every order its actors can take (no GPU needed).

An mbarrier tells a waiter only the parity of the phase it is in.  A wait for
phase k is right while k + 1 phases are complete; it passes too early where k - 1
are (the parity is the same) and is lost where k + 2 are: the waiter then waits
for a phase that may need its own arrival.  The model holds one tile with the
kernel's two score buffers: the issuer queues products and commits in the order
of the kernel, the tensor core ends them in order, each softmax warp waits for
the scores of every step, arrives with its weights, and waits for both buffers'
last products at a unit's end."""
import pytest

WARPS = 2                                  # arrivals a p_ready phase needs (four in the kernel)
COUNT = {"s0": 1, "s1": 1, "p0": WARPS, "p1": WARPS, "seen": WARPS}


def issuer(units, handshake):
    """One entry per step: ("wait", barrier, phase) or ("commit", barrier)."""
    ops, p = [], 0
    for u, n in enumerate(units):
        if handshake and u > 0:
            ops.append(("wait", "seen", u - 1))
        ops += [("commit", "s0"), ("commit", "s1")]        # S = Q K^T of the first tile
        for _ in range(n):
            for hf in "01":
                ops += [("wait", "p" + hf, p), ("commit", "s" + hf)]   # O += P V and the next S
            p += 1
    return ops


def softmax(units, handshake):
    ops, s = [], 0
    for n in units:
        for _ in range(n):
            for hf in "01":
                ops += [("wait", "s" + hf, s), ("arrive", "p" + hf)]
            s += 1
        ops += [("wait", "s0", s), ("wait", "s1", s)]      # the unit's last products
        s += 1
        if handshake:
            ops.append(("arrive", "seen"))
    return ops


def walk(units, handshake):
    """(orders that lose a wait or pass one early, whether every order ends)."""
    actors = [issuer(units, handshake)] + [softmax(units, handshake)] * WARPS
    commits = [b for op, b, *_ in actors[0] if op == "commit"]
    issued = [0]                                           # commits before each issuer step
    for op in actors[0]:
        issued.append(issued[-1] + (op[0] == "commit"))
    before = [{}]                                          # arrivals before each softmax step
    for op in actors[1]:
        d = dict(before[-1])
        if op[0] == "arrive":
            d[op[1]] = d.get(op[1], 0) + 1
        before.append(d)

    def phases(bar, state):
        pcs, ended = state[:-1], state[-1]
        n = commits[:ended].count(bar) if bar[0] == "s" and bar != "seen" else \
            sum(before[pc].get(bar, 0) for pc in pcs[1:])
        return n // COUNT[bar]

    start = (0,) * (1 + WARPS) + (0,)
    todo, known, wrong, stuck = [start], {start}, 0, 0
    while todo:
        st = todo.pop()
        nexts = []
        if st[-1] < issued[st[0]]:                         # the tensor core ends a product
            nexts.append(st[:-1] + (st[-1] + 1,))
        for a, ops in enumerate(actors):
            if st[a] == len(ops):
                continue
            op = ops[st[a]]
            if op[0] == "wait":
                done, k = phases(op[1], st), op[2]
                passes = (done & 1) != (k & 1)
                if done >= k + 2 or (passes and done <= k):
                    wrong += 1
                if not passes:
                    continue
            nexts.append(st[:a] + (st[a] + 1,) + st[a + 1:])
        if not nexts and any(st[a] < len(ops) for a, ops in enumerate(actors)):
            stuck += 1
        for n in nexts:
            if n not in known:
                known.add(n)
                todo.append(n)
    return wrong, stuck


@pytest.mark.parametrize("units", [(1, 1), (1, 2, 1), (2, 1, 1), (3, 2)])
def test_no_order_loses_a_phase(units):
    assert walk(units, True) == (0, 0)


def test_without_the_issuers_wait_a_late_warp_is_lapped():
    wrong, stuck = walk((1, 1), False)
    assert wrong > 0 and stuck > 0
