"""Plant plausible mistakes in copies of the 4-bit oracle (oracle/int4.py) and
check that its pins catch each one (CPU only)."""
import os
import types

import pytest

import oracle
import test_oracle_int4 as P

FILE = os.path.join(os.path.dirname(oracle.__file__), "int4.py")

MUTANTS = [
    ("sixteen steps", "s, z = ((hi - lo) / 15.0)", "s, z = ((hi - lo) / 16.0)"),
    ("codes truncated", "np.rint(u)", "np.floor(u)"),
    ("no clipping", "        y = np.clip(y, -t, t)\n", "        pass\n"),
    ("clipped from above only", "np.clip(y, -t, t)", "np.minimum(y, t)"),
    ("division by a zero scale", "np.where(sf > 0, (y - zf) / np.where(sf > 0, sf, 1.0), 0.0)", "(y - zf) / np.where(sf > 0, sf, 1e-30)"),
    ("nibbles swapped", "4 * group + (index % 8) // 2, 4 * (p % 2)", "4 * group + (index % 8) // 2, 4 - 4 * (p % 2)"),
    ("K group and chunk exchanged", "16 * (index // 8) + 4 * group", "16 * group + 4 * (index // 8)"),
    ("V codes behind a half without pairs", "    return half + (p // 2) * 64 + t", "    return 4096 + (p // 2) * 64 + t"),
    ("V pairs in K's place", "base = 4096 + which * (4096 + 256 * ng)", "base = 4096 + which * 256 * ng"),
    ("values without zero", "return codes * p[..., 0] + p[..., 1]", "return codes * p[..., 0]"),
    ("scale and zero swapped", "return codes * p[..., 0] + p[..., 1]", "return codes * p[..., 1] + p[..., 0]"),
    ("one group's pair everywhere", "np.repeat(pairs.astype(np.float64), g, axis=1)", "np.tile(pairs.astype(np.float64), (1, g, 1))"),
    ("2-bit codes read with four bits", "(3 if bits == 2 else 15)", "15"),
    ("stored over the neighbour's nibble", "(0xF0 if nib == 0 else 0x0F)", "0"),
    ("mapped back by R", "vs @ R[kv][1].T", "vs @ R[kv][1]"),
    ("softmax scale dropped", "x = sm_scale * (k @ q[b, h])", "x = k @ q[b, h]"),
    ("window left out", "v = np.concatenate([vs @ R[kv][1].T, bf16_kv[b, :m, kv, 1]])", "v = np.concatenate([vs @ R[kv][1].T, 0 * bf16_kv[b, :m, kv, 1]])"),
    ("kept token's pair left behind", "out[d0 + da] = pool[s0 + sa]\n                    sa = np.unique", "sa = np.unique"),
    ("gathered from the list's index", "x = int(keep[b, i])", "x = i"),
]


def pins():
    """Every pin with its parameters, as calls."""
    for name in dir(P):
        f = getattr(P, name)
        if not name.startswith("test_"):
            continue
        marks = [m for m in getattr(f, "pytestmark", []) if m.name == "parametrize"]
        for v in marks[0].args[1] if marks else [None]:
            yield name, (lambda f=f, v=v: f() if v is None else f(v))


def run(monkeypatch, text):
    mod = types.ModuleType("oracle.int4_mutant")
    mod.__file__ = FILE
    exec(compile(text, FILE, "exec"), mod.__dict__)
    monkeypatch.setattr(P, "I", mod)
    failed = []
    for name, call in pins():
        try:
            call()
        except Exception:
            failed.append(name)
    return failed


def test_pins_hold_for_the_oracle_itself(monkeypatch):
    with open(FILE, encoding="utf-8") as f:
        assert run(monkeypatch, f.read()) == []


@pytest.mark.filterwarnings("ignore")
@pytest.mark.parametrize("what,a,b", MUTANTS, ids=[m[0] for m in MUTANTS])
def test_a_planted_mistake_fails_a_pin(monkeypatch, what, a, b):
    with open(FILE, encoding="utf-8") as f:
        text = f.read()
    assert text.count(a) == 1
    assert run(monkeypatch, text.replace(a, b)) != []
