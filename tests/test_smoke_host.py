"""The smoke's decode batches run both forms of the 4-bit product, by the rule in
its source and the batches' sizes."""
import ast
import os
import re

from test_warp_convergence_host import code

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def sizes():
    """K, E, H, I and the tokens of _smoke_decode."""
    with open(os.path.join(ROOT, "__graft_entry__.py")) as f:
        tree = ast.parse(f.read())
    body = next(n for n in tree.body if isinstance(n, ast.FunctionDef) and n.name == "_smoke_decode")
    first = next(n for n in ast.walk(body) if isinstance(n, ast.Assign) and isinstance(n.targets[0], ast.Tuple))
    assert [t.id for t in first.targets[0].elts] == ["K", "E", "H", "I"]
    loop = next(n for n in ast.walk(body) if isinstance(n, ast.For) and getattr(n.target, "id", "") == "T")
    return (*ast.literal_eval(first.value), ast.literal_eval(loop.iter))


def test_both_forms_run():
    rule = re.search(r"mean <= (\d+) \|\| \(mean <= (\d+) && weights <= \(1ll << (\d+)\)\) \|\| "
                     r"\(mean <= (\d+) && weights <= \(1ll << (\d+)\)\)", code("grouped_w4.cu"))
    any_weights, some, some_bits, more, more_bits = map(int, rule.groups())
    K, E, H, I, batches = sizes()  # noqa: E741

    def few(T, N, Kd):
        live = min(E, T * K)
        mean, weights = -(-T * K // live), live * N * Kd
        return mean <= any_weights or (mean <= some and weights <= 1 << some_bits) or \
            (mean <= more and weights <= 1 << more_bits)

    forms = [[few(T, N, Kd) for N, Kd in ((2 * I, H), (H, I))] for T in batches]
    assert forms == [[True, True], [False, False]]
