"""Which tokens count in the balance loss when logits are not numbers.

A token has no choice, and does not count, only if every one of its E logits is -inf.  A NaN is not
-inf: such a token counts, alone or beside experts that cannot be chosen, at every E, whether its row
fills its lanes or not.  Then lse, its gradient row and the losses are NaN, and the other tokens'
gradients are what they are without it but for the counts.  Bounds as for finite logits."""
import numpy as np
import pytest
import torch

from oracle import block_ref as R
from block_testlib import f64
from test_gpu_balance import check, make, run

NAN, INF = np.nan, np.inf


def spoil(row, kind):
    """One token's logits with a value that is not finite."""
    row = row.copy()
    E = row.size
    at = E // 2
    if kind == "one_nan":
        row[at] = NAN
    elif kind == "all_nan":
        row[:] = NAN
    elif kind == "nan_beside_forbidden":
        row[:] = -INF
        row[at] = NAN
    elif kind == "half_nan_half_forbidden":
        row[:] = -INF
        row[::2] = NAN
    elif kind == "inf":
        row[at] = INF
    elif kind == "inf_beside_forbidden":
        row[:] = -INF
        row[at] = INF
    elif kind == "nan_beside_inf":
        row[0], row[at] = NAN, INF
    else:
        raise KeyError(kind)
    return row


KINDS = ("one_nan", "all_nan", "nan_beside_forbidden", "half_nan_half_forbidden", "inf", "inf_beside_forbidden",
         "nan_beside_inf")


@pytest.mark.parametrize("kind", KINDS)
def test_oracle_counts_every_row_but_one_of_forbidden_experts(kind):
    rng = np.random.default_rng(1)
    T, E, k = 9, 8, 2
    logits = rng.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :k].astype(np.int32)
    logits[4] = spoil(logits[4], kind)
    logits[6] = -INF
    with np.errstate(invalid="ignore"):
        b = R.balance(logits, ids)
        d, _ = R.balance_grad(b, k, (0.5, 0.25))
    assert b["tokens"].tolist() == [T - 1, T - 1, 1] and b["counts"].sum() == k * (T - 1)
    assert np.isnan(b["losses"]).all() and np.isnan(b["lse"][4]) and b["lse"][6] == -INF
    assert np.isnan(d[4]).all() and np.isfinite(np.delete(d, 4, 0)).all() and not d[6].any()


# one launch (one tile), several tiles, and groups with a mask; every layout of a row, filled and not
LAYOUTS = [8, 16, 32, 60, 64, 7, 65, 96, 128, 160, 256, 384, 385, 512, 513, 1000, 1023, 1024]


@pytest.mark.gpu
@pytest.mark.parametrize("E", LAYOUTS)
@pytest.mark.parametrize("T,S", [(50, 1), (300, 1), (300, 3)])
def test_tokens_that_are_not_numbers_count(T, S, E):
    for i, kind in enumerate(KINDS):
        print(f"[case] balance {kind} T={T} S={S} E={E}", flush=True)
        c = make(T, E, min(4, E), 40 + i, S=S, mask=S > 1)
        if S > 1:
            c["mask"][[3, T - 2]] = 1
            c["offsets"] = np.array([0, T // 3, T // 2, T], np.int32)
        for t in (3, T - 2):   # in the first and in the last group
            c["logits"][t] = spoil(np.random.default_rng(t).standard_normal(E).astype(np.float32), kind)
        c["logits"][T // 2] = -INF
        if S > 1:
            c["mask"][T // 2] = 1
        o = run(c)
        with np.errstate(invalid="ignore"):
            check(c, o)
        lse = f64(o["lse"])
        assert np.isnan(lse[[3, T - 2]]).all() and lse[T // 2] == -INF
        assert np.isnan(f64(o["losses"])).all()
        assert torch.isnan(o["d_logits"][3]).all()
