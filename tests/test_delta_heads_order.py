"""The tensor-memory places of the delta rule's walk of whole heads (delta_heads.cu), as a model on the CPU.

MMAs that are in flight at the same time are ordered among themselves only if they have the same accumulator and the same
shape.  So of two that touch the same columns, one of them writing, either they are of that kind and issued by one
thread, or the first is known to be complete (its commit has been waited for) before the second is issued.  The MMAs are
taken from the kernel's source: accumulator, left operand and shape of each call in its loops, with the constants as they
stand there."""
import os
import re

import pytest

import moe_expert_step_gb300 as ms

SOURCE = os.path.join(os.path.dirname(ms.__file__), "csrc", "delta_heads.cu")
PRODUCTS = ["keys", "queries", "new", "outputs", "state"]  # in the order of the source; what is waited for between them:
WAITED = {"keys": set(), "queries": {"keys"}, "new": {"keys"}, "outputs": {"keys", "queries", "new"},
          "state": {"keys", "queries", "new"}}  # (the products of the chunk before are all complete)
ISSUER = {p: 1 if p == "queries" else 0 for p in PRODUCTS}


def python(expr):
    """A C++ expression of sums, products and conditionals as a Python one."""
    expr = re.sub(r"\bconstexpr\b", "", expr)
    while "?" in expr:
        new = re.sub(r"([\w ><=]+?) \? ([\w() +*]+?) : ([\w() +*-]+?)(?=[),]|$)", r"(\2) if \1 else (\3)", expr)
        assert new != expr, expr
        expr = new
    return expr


def arguments(text, at):
    """The arguments of a call whose opening bracket is at `at`."""
    depth, args, start = 0, [], at + 1
    for i in range(at, len(text)):
        depth += (text[i] == "(") - (text[i] == ")")
        if (text[i] == "," and depth == 1) or depth == 0:
            args.append(text[start:i].strip())
            start = i + 1
        if depth == 0:
            return args


def mmas(text, DK):
    """[(product, first accumulator column, columns, first operand column, accumulates)] in the order of their issue."""
    env = {m: int(v) for m, v in re.findall(r"constexpr uint32_t (k\w) = (\d+);", text)}
    later = re.search(r"constexpr uint32_t later\(int kt\) \{ return (.+?); \}", text)
    if later:
        parts = [python(x) for x in re.findall(r"\(([^()]+)\)", later.group(1))]
        assert later.group(1).startswith("kM + ")
        env["later"] = lambda kt: env["kM"] + sum(eval(x, {"kt": kt}) for x in parts)
    body = text[text.index("delta_heads_kernel(const DeltaArgs"):]
    calls = [[arguments(body, m.end() - 1), body.rfind("for (int kt", 0, m.start())] for m in
             re.finditer(r"tc::mma_f16_tmem_a\(", body)]
    loops = sorted({at for _, at in calls})
    assert len(loops) == len(PRODUCTS)
    out = []
    for product, at in zip(PRODUCTS, loops):
        steps = DK // 16 if product in ("keys", "queries") else 4
        local = dict(env, tmem=0, DK=DK)
        inner = body[at:body.index("tc::mma_commit", at)]
        d = re.search(r"\bd = (.+);", inner)
        for kt in range(steps):
            local["kt"] = kt
            if d:
                local["d"] = eval(python(d.group(1)), {}, local)
            n = DK if product == "state" else 64 if product in ("keys", "queries") else 64 - 16 * kt
            for args, loop in calls:
                if loop == at:
                    acc, a = (eval(python(x), {}, local) for x in args[:2])
                    out.append((product, acc, n, a, bool(eval(python(args[4]), {}, local))))
    return out


def conflicts(ops):
    found = []
    for j, (p, acc, n, a, _) in enumerate(ops):
        for q, acc0, n0, a0, _ in ops[:j]:
            if q in WAITED[p]:
                continue
            overlap = lambda x, nx, y, ny: x < y + ny and y < x + nx  # noqa: E731
            if overlap(acc, n, acc0, n0) and not (acc == acc0 and n == n0 and ISSUER[p] == ISSUER[q]):
                found.append((p, q, "accumulators", acc, acc0))
            if overlap(acc, n, a0, 8):
                found.append((p, q, "writes an operand", acc, a0))
            if overlap(a, 8, acc0, n0):
                found.append((p, q, "reads an accumulator", a, acc0))
    return found


@pytest.mark.parametrize("DK", [64, 128])
def test_products_in_flight_have_places_of_their_own(DK):
    ops = mmas(open(SOURCE).read(), DK)
    assert len(ops) == 2 * DK // 16 + DK // 16 + 12 + 4 + 8
    assert conflicts(ops) == []
    columns = int(re.search(r"kColumns = (\d+);", open(SOURCE).read()).group(1))
    assert columns <= 512 and all(acc + n <= columns and a + 8 <= columns for _, acc, n, a, _ in ops)


@pytest.mark.parametrize("DK", [64, 128])
def test_every_token_gets_every_product_once(DK):
    """The sums that the threads form: token 16 p + i of the first accumulator and of those of sixteens up to p; the first
    product into each accumulator, and only that, begins a sum (the outputs' first one adds to what the threads wrote)."""
    ops = mmas(open(SOURCE).read(), DK)
    for product, each in (("new", 3), ("outputs", 1)):
        mine = [o for o in ops if o[0] == product]
        by_acc = {}
        for kt in range(4):
            group = mine[kt * each:(kt + 1) * each]
            assert len({o[1] for o in group}) == 1 and {o[2] for o in group} == {64 - 16 * kt}
            by_acc[group[0][1]] = group
            begins = [not o[4] for o in group]
            assert begins == [product == "new" or kt > 0] + [False] * (each - 1)
        assert len(by_acc) == 4
    for product in ("keys", "queries", "state"):
        assert [not o[4] for o in ops if o[0] == product][:1] == [True]
        assert all(o[4] for o in [o for o in ops if o[0] == product][1:])


def test_the_model_finds_shared_places():
    """Sums of several shapes in one place, and an accumulator over another product's operand, are found."""
    ops = [("new", 64 + 16 * kt, 64 - 16 * kt, 128 + 8 * kt, kt > 0) for kt in range(4)]
    assert any(f[2] == "accumulators" for f in conflicts(ops))
    ops = [("outputs", 0, 64, 128, True), ("state", 128, 128, 64, False)]
    assert [f[2] for f in conflicts(ops)] == ["writes an operand"]
    ops = [("keys", 128, 64, 0, False), ("keys", 128, 64, 64, True)]
    assert conflicts(ops) == []
