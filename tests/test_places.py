"""What a call writes must lie apart from what it reads: the host's arithmetic of
places, and the refusals of the losses' entries (before any CUDA call)."""
import ctypes
import os
import subprocess

import pytest

import test_losses_abi as abi
from conftest import ROOT
from test_losses_abi import BF16, EINVAL, i64, lib, vp   # noqa: F401 (lib: a fixture)

SRC = os.path.join(ROOT, "tests", "host_model", "places_test.cpp")
OUT = os.path.join(ROOT, "tests", "_build")


def test_overlaps_on_host():
    os.makedirs(OUT, exist_ok=True)
    exe = os.path.join(OUT, "places")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-o", exe, SRC])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "failures=0" in r.stdout, r.stdout + r.stderr


# vectors of a call, each a place of its own that is never read: every call here is refused first
MIB = 1 << 20
N = 100


def at(k):
    return (k + 1) * MIB


def calls(lib, **moved):   # noqa: F811
    """What the entries say to vectors at their own places, some of them moved."""
    def p(name, k):
        return moved.get(name, at(k))
    n, pairs = moved.get("n", N), 3
    policy = abi.policy(old_logps=p("old_logps", 0), advantages=p("advantages", 1), weights=p("weights", 2), ref_logps=p("ref_logps", 3))
    preference = abi.preference()
    logps, out, loss, stats, scratch = (vp(p(name, 4 + k)) for k, name in enumerate(("logps", "out", "loss", "stats", "scratch")))
    yield "policy", lambda: lib.seqsum_policy_loss(logps, i64(n), policy, out, loss, stats, scratch, None)
    yield "backward", lambda: lib.seqsum_policy_loss_backward(logps, i64(n), policy, vp(p("dloss", 9)), out, None)
    # 100 rows of 50 16-bit numbers, 80 from one to the next
    yield "rows", lambda: lib.seqsum_token_policy_grad(
        vp(p("logits", 10)), ctypes.c_int32(BF16), i64(n), i64(50), i64(moved.get("stride", 80)), vp(p("tokens", 11)), policy,
        vp(p("dlogits", 12)), i64(moved.get("dstride", 80)), vp(p("lp", 13)), vp(p("entropies", 14)), loss, stats, scratch, None)
    offsets, scores, slopes, losses = (vp(p(name, 15 + k)) for k, name in enumerate(("offsets", "scores", "slopes", "losses")))
    yield "preference", lambda: lib.seqsum_preference_loss(
        logps, vp(p("ref_logps", 3)), vp(p("weights", 2)), i64(n), offsets, i64(pairs), preference, out, loss, scores, slopes,
        losses, None)
    yield "preference_backward", lambda: lib.seqsum_preference_backward(
        vp(p("weights", 2)), i64(n), offsets, i64(pairs), slopes, vp(p("dloss", 9)), out, None)


ENDS = dict(old_logps=(0, 4 * N), advantages=(1, 4 * N), weights=(2, 4 * N), ref_logps=(3, 4 * N), logps=(4, 4 * N), out=(5, 4 * N),
            loss=(6, 4), stats=(7, 24), dloss=(9, 4), logits=(10, 2 * (99 * 80 + 50)), tokens=(11, 8 * N),
            dlogits=(12, 2 * (99 * 80 + 50)), lp=(13, 4 * N), entropies=(14, 4 * N), offsets=(15, 56), scores=(16, 24),
            slopes=(17, 24), losses=(18, 12))
VECTORS = ("old_logps", "advantages", "weights", "ref_logps")
# what is written, and what it must not lie in
APART = dict(policy=[("out", (*VECTORS, "loss", "stats")), ("loss", (*VECTORS, "logps", "stats")), ("stats", (*VECTORS, "logps"))],
             backward=[("out", (*VECTORS, "dloss"))],
             rows=[(w, (*VECTORS, "tokens", "logits", *others)) for w, others in (
                 ("lp", ("dlogits", "entropies", "loss", "stats")), ("entropies", ("dlogits", "loss", "stats")),
                 ("loss", ("dlogits", "stats")), ("stats", ("dlogits",)))] + [("dlogits", (*VECTORS, "tokens"))],
             preference=[("out", ("ref_logps", "weights", "offsets", "loss", "scores", "slopes", "losses")),
                         ("loss", ("logps", "ref_logps", "weights", "offsets", "scores", "slopes", "losses")),
                         ("scores", ("logps", "ref_logps", "weights", "offsets", "slopes", "losses")),
                         ("slopes", ("logps", "ref_logps", "weights", "offsets", "losses")),
                         ("losses", ("logps", "ref_logps", "weights", "offsets"))],
             preference_backward=[("out", ("weights", "offsets", "slopes", "dloss"))])


@pytest.mark.parametrize("entry,written,other", [(e, w, o) for e, ws in APART.items() for w, os_ in ws for o in os_])
def test_overlapping_places_refused(lib, entry, written, other):   # noqa: F811
    place, size = ENDS[other]
    unit = 8 if other in ("tokens", "offsets") else 2 if other in ("logits", "dlogits") else 4
    align = 2 if written == "dlogits" else 4
    mine = ENDS[written][1]
    # at the same place, at the other's last number, and beginning before it, its last one there
    for address in {at(place), (at(place) + size - unit) // align * align, at(place) - mine + align}:
        assert dict(calls(lib, **{written: address}))[entry]() == EINVAL, (entry, written, other, address - at(place))


@pytest.mark.parametrize("entry,written", [("policy", "out"), ("backward", "out"), ("preference", "out"), ("rows", "dlogits")])
def test_only_the_very_place_is_in_place(lib, entry, written):   # noqa: F811
    """The gradient may be the very numbers that it is of, not some of them and not their rows at another stride."""
    of = "logits" if entry == "rows" else "logps"
    for shift in (-4, 4, 40, 4 * N - 4):
        assert dict(calls(lib, **{written: at(ENDS[of][0]) + shift}))[entry]() == EINVAL
    if entry == "rows":
        assert dict(calls(lib, dlogits=at(ENDS["logits"][0]), dstride=96))[entry]() == EINVAL
        assert dict(calls(lib, dlogits=at(ENDS["logits"][0]) + 98, dstride=80))[entry]() == EINVAL   # the last of a row's numbers
        assert dict(calls(lib, lp=at(ENDS["logits"][0]) + 160 * 40 + 96))[entry]() == EINVAL


def test_scratch_that_is_used(lib):   # noqa: F811
    n = 65537
    k = dict(n=n, old_logps=1 << 30, advantages=2 << 30, weights=3 << 30, ref_logps=None, logps=4 << 30, out=5 << 30,
             logits=6 << 30, tokens=7 << 30, dlogits=8 << 30, lp=9 << 30, entropies=10 << 30)
    for entry, places in (("policy", (1, 2, 3, 4, 5)), ("rows", (1, 2, 3, 6, 7, 8, 9, 10))):
        for g in places:
            for address in (g << 30, (g << 30) - 49152 + 8, (g << 30) + 4 * n - 4 - 4 * n % 8):
                assert dict(calls(lib, **k, scratch=address))[entry]() == EINVAL, (entry, g)


# The refusals of settings and vectors again, where all vectors lie apart: what is refused is the setting or the vector.
APART_POLICY = dict(old_logps=at(0), advantages=at(1), weights=at(2), ref_logps=at(3))
APART_VALUE = dict(zip(("logps", "dlogps", "loss", "stats", "scratch"), (vp(at(4 + k)) for k in range(5))))
APART_BACKWARD = dict(logps=vp(at(4)), dlogps=vp(at(5)), dloss=vp(at(9)))
APART_ROWS = dict(zip(("logits", "tokens", "d", "logps", "entropies", "loss", "stats", "scratch"), (vp(at(10 + k)) for k in range(8))))
APART_PAIRS = dict(zip(("logps", "ref", "weights", "offsets", "dlogps", "loss", "scores", "slopes", "losses"),
                       (vp(at(k)) for k in range(9))))


def odd(address):
    """The same misplacement, at a place of its own."""
    return at(30) + address % MIB if isinstance(address, int) else None if address is None else vp(at(30) + address.value % MIB)


def moved(bad):
    return {k: odd(v) if isinstance(v, vp) or v is None else v for k, v in bad.items()}


@pytest.mark.parametrize("bad", abi.BAD_POLICIES)
def test_policies_apart(lib, bad):   # noqa: F811
    s = abi.policy(**{**APART_POLICY, **{k: odd(v) if k in APART_POLICY else v for k, v in bad.items()}})
    assert abi.value(lib, s, **APART_VALUE) == abi.backward(lib, s, **APART_BACKWARD) == abi.rows(lib, s, **APART_ROWS) == EINVAL


def bad_of(test):
    """What an earlier test is parametrised by."""
    return next(m.args[1] for m in test.pytestmark if m.name == "parametrize")


@pytest.mark.parametrize("bad", bad_of(abi.test_settings_of_rows_refused))
def test_settings_of_rows_apart(lib, bad):   # noqa: F811
    assert abi.rows(lib, abi.policy(**APART_POLICY, **bad), **APART_ROWS) == EINVAL


@pytest.mark.parametrize("bad", bad_of(abi.test_tokens_refused))
def test_tokens_apart(lib, bad):   # noqa: F811
    assert abi.value(lib, abi.policy(**APART_POLICY), **{**APART_VALUE, **moved(bad)}) == EINVAL


@pytest.mark.parametrize("bad", bad_of(abi.test_backward_refused))
def test_backward_apart(lib, bad):   # noqa: F811
    assert abi.backward(lib, abi.policy(**APART_POLICY), **{**APART_BACKWARD, **moved(bad)}) == EINVAL


@pytest.mark.parametrize("bad", [b for b in bad_of(abi.test_rows_refused) if not any(v in (abi.P, abi.Q) for v in b.values())
                                 and not ("logps" in b and "entropies" in b)])
def test_rows_apart(lib, bad):   # noqa: F811
    assert abi.rows(lib, abi.policy(**APART_POLICY), **{**APART_ROWS, **moved(bad)}) == EINVAL


@pytest.mark.parametrize("bad", bad_of(abi.test_preferences_refused))
def test_preferences_apart(lib, bad):   # noqa: F811
    assert abi.pairs(lib, abi.preference(**bad), **APART_PAIRS) == EINVAL


@pytest.mark.parametrize("bad", bad_of(abi.test_pairs_refused))
def test_pairs_apart(lib, bad):   # noqa: F811
    assert abi.pairs(lib, abi.preference(), **{**APART_PAIRS, **moved(bad)}) == EINVAL


@pytest.mark.parametrize("bad", bad_of(abi.test_preference_backward_refused))
def test_preference_backward_apart(lib, bad):   # noqa: F811
    a = {**dict(weights=vp(at(0)), n=100, offsets=vp(at(1)), k=3, slopes=vp(at(2)), dloss=vp(at(3)), dlogps=vp(at(4))), **moved(bad)}
    assert lib.seqsum_preference_backward(a["weights"], i64(a["n"]), a["offsets"], i64(a["k"]), a["slopes"], a["dloss"],
                                          a["dlogps"], None) == EINVAL
