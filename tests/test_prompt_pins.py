"""Pins of the oracles for appended rows and the counted page pool, and the
refusals of their Python entry points (CPU only)."""
import types

import numpy as np
import pytest
import torch

import oracle.append_ref as ar
import oracle.page_pool_ref as pp
from paged_mla_speculative_gb300 import binding as mb


def test_rotation_is_a_turn_of_each_pair():
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal(64), rng.uniform(0, 6, 32)
    cs = np.concatenate([np.cos(angle), np.sin(angle)])
    for halves in (False, True):
        y = ar.rotate(x, cs, halves)
        a = x[:32] + 1j * x[32:] if halves else x[0::2] + 1j * x[1::2]
        b = y[:32] + 1j * y[32:] if halves else y[0::2] + 1j * y[1::2]
        assert np.allclose(b, a * np.exp(1j * angle))
    # the product of a query and a key depends on the distance alone
    z = rng.standard_normal(64)
    turn = lambda v, p: ar.rotate(v, np.concatenate([np.cos(p * angle), np.sin(p * angle)]), False)  # noqa: E731
    assert np.isclose(turn(x, 3) @ turn(z, 8), turn(x, 10) @ turn(z, 15))


def test_append_hand_case():
    kv = np.zeros((4, 576))
    kv[:, 0], kv[:, 512] = 2.0, 5.0
    w = np.full(512, 3.0)
    cs = np.zeros((2, 64))
    cs[0, :32] = 1.0                                # position 0: no turn
    cs[1, 32:] = 1.0                                # position 1: a quarter
    cache, q = np.full((6, 576), -1.0), np.full((4, 1, 576), -2.0)
    pe = np.zeros((4, 1, 64))
    pe[:, 0, 2] = 7.0
    out, qq, flags = ar.append_kv(kv, w, 0.0, None, pe, cs, [0, 1, 9, 0], [4, 2, 0, -1], False, cache, q)
    root = np.sqrt(4.0 / 512)
    assert np.isclose(out[4, 0], 6.0 / root) and out[4, 512] == 5.0 and out[4, 513] == 0.0
    assert out[2, 512] == 0.0 and out[2, 513] == 5.0
    assert (out[[0, 1, 3, 5]] == -1).all() and flags == ar.BAD_POS
    assert qq[0, 0, 514] == 7.0 and qq[1, 0, 515] == 7.0 and (qq[:2, 0, :512] == -2).all()
    assert (qq[2:] == -2).all()


def _pool():
    # 10 pages; request 0: 150 rows on pages 3 1 4, request 1: 64 rows on 9.
    rows = [f"r{s}" for s in range(640)]
    refs = [0, 1, 0, 1, 1, 0, 0, 0, 0, 1]
    return [3, 1, 4, 9], [0, 3, 4], [150, 64], refs, [0, 2, 5, 6, 7, 8], rows


class _Rows(list):
    """Rows as numbers; rows[0] * 0 is the zero row."""


def test_fork_and_free_hand_case():
    idx, ptr, lens, refs, stack, _ = _pool()
    cache = _Rows(range(640))
    t, ln, refs2, stack2, flags = pp.fork_kv([0, 1, 0], idx, ptr, lens, [cache], refs, stack, 8, 100, 1000)
    assert t == [[3, 1, 8], [9, 7], [3, 1, 6]] and ln == [158, 72, 158] and flags == 0
    assert stack2 == [0, 2, 5]
    assert refs2 == [0, 3, 0, 3, 1, 0, 1, 1, 1, 2]
    assert cache[8 * 64:8 * 64 + 22] == list(range(4 * 64, 4 * 64 + 22)) and cache[8 * 64 + 22] == 8 * 64 + 22
    assert cache[6 * 64:6 * 64 + 22] == list(range(4 * 64, 4 * 64 + 22)) and cache[7 * 64] == 7 * 64
    # request 0 itself and one of its children end: page 4 and the child's own
    refs3, stack3, flags = pp.free_kv([[3, 1, 4], [3, 1, 8]], refs2, stack2)
    assert refs3 == [0, 1, 0, 1, 0, 0, 1, 1, 0, 2] and stack3 == [0, 2, 5, 4, 8] and flags == 0
    # freed twice, and a page that is none
    refs4, stack4, flags = pp.free_kv([[4, 77]], refs3, stack3)
    assert refs4 == refs3 and stack4 == stack3 and flags == pp.BAD_REF | pp.BAD_SLOT


def test_fork_cuts_the_run_that_does_not_fit():
    idx, ptr, lens, refs, stack, _ = _pool()
    cache = _Rows(range(640))
    # two fresh pages: child 2 and everything after it get none, a child of
    # full pages only among them
    t, ln, refs2, left, flags = pp.fork_kv([0, 0, 0, 1], idx, ptr, lens, [cache], refs, [0, 2], 0, 100, 1000)
    assert [len(x) for x in t] == [3, 3, 0, 0] and ln == [150, 150, 0, 0] and left == [] and flags == pp.CAPACITY
    t, ln, _, left, flags = pp.fork_kv([0, 0], idx, ptr, lens, [cache], refs, stack, 0, 5, 1000)
    assert [len(x) for x in t] == [3, 0] and flags == pp.CAPACITY
    t, ln, _, left, flags = pp.fork_kv([5, 0, 1], idx, ptr, [-1, 64], [cache], refs, stack, 0, 5, 1000)
    assert t == [[], [], [9]] and left == stack and flags == pp.BAD_POOL | pp.BAD_LEN


def _stub(**kw):
    return types.SimpleNamespace(torch_device=torch.device("cpu"), num_slots=128, H=2, max_kv_len=100, page_size=64,
                                 T=4, out_dtype=torch.float32, handle=None, **kw)


def test_append_refuses_what_it_cannot_read():
    bf, i32 = torch.bfloat16, torch.int32
    ok = dict(kv=torch.zeros(3, 576, dtype=bf), weight=torch.zeros(512, dtype=bf), eps=1e-6, cos_sin=torch.zeros(8, 64),
              positions=torch.zeros(3, dtype=i32), slots=torch.zeros(3, dtype=i32),
              kv_cache=torch.zeros(128, 576, dtype=bf), q_pe=torch.zeros(3, 2, 64, dtype=bf),
              q_nope=torch.zeros(3, 2, 512, dtype=bf))
    wrong = [(TypeError, dict(kv=torch.zeros(3, 576))), (ValueError, dict(kv=torch.zeros(3, 580, dtype=bf)[:, :576])),
             (ValueError, dict(kv=torch.zeros(2, 576, dtype=bf))), (ValueError, dict(kv=torch.zeros(576, 3, dtype=bf).t())),
             (TypeError, dict(weight=torch.zeros(512))), (ValueError, dict(cos_sin=torch.zeros(8, 32))),
             (TypeError, dict(positions=torch.zeros(3, dtype=torch.int64))), (ValueError, dict(slots=torch.zeros(4, dtype=i32))),
             (ValueError, dict(kv_cache=torch.zeros(64, 576, dtype=bf))), (ValueError, dict(q_pe=torch.zeros(3, 3, 64, dtype=bf))),
             (ValueError, dict(q_pe=None)), (ValueError, dict(q_nope=None)),
             (TypeError, dict(q=torch.zeros(3, 2, 576)))]
    for err, over in wrong:
        with pytest.raises(err):
            mb.append_kv(_stub(), **{**ok, **over})


def test_pool_calls_refuse_what_they_cannot_read():
    i32 = torch.int32
    z = lambda n: torch.zeros(n, dtype=i32)  # noqa: E731
    ok = dict(parents=z(3), kv_indices=z(4), kv_indptr=z(3), kv_lens=z(2), kv_cache=torch.zeros(128, 576, dtype=torch.bfloat16),
              page_refs=z(2), free_pages=z(2), free_count=z(1))
    wrong = [(TypeError, dict(parents=torch.zeros(3))), (ValueError, dict(kv_indptr=z(2))), (ValueError, dict(page_refs=z(3))),
             (ValueError, dict(free_pages=z(1))), (ValueError, dict(free_count=z(2))),
             (ValueError, dict(kv_cache=torch.zeros(2, 64, 576, dtype=torch.bfloat16))), (ValueError, dict(child_lens=z(2)))]
    for err, over in wrong:
        with pytest.raises(err):
            mb.fork_kv(_stub(), **{**ok, **over})
    with pytest.raises(ValueError):
        mb.free_kv(_stub(), z(4), z(3), z(3), z(2), z(1))


def test_null_plans_are_refused():
    lib = mb.load_library()
    assert lib.mla_verify_append_kv(None, 0, None, 0, None, 0.0, None, 0, 0, None, 0, 0, None, 0, None, None, 0, None, None,
                                    None) == -1
    assert lib.mla_verify_fork_kv(None, 1, None, 1, None, None, None, None, 1, 0, 0, None, None, None, None, 0, None, None,
                                  None) == -1
    assert lib.mla_verify_free_kv(None, 1, None, None, None, None, None, None) == -1
