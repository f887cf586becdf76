"""A step's page map taken back: with state_out apart from state_in, what state_in
counts is as it was, and the step can be mapped again with other new_lens.  So
the beams of a group are granted together or not at all."""
import numpy as np
import pytest

from oracle import decode_step as ref

PS, MP, W, GROUPS = 4, 6, 4, 5
B, P = W * GROUPS, 72


def start(seed):
    """Groups of beams of equal lengths, in a pool that cannot serve all of them."""
    rng = np.random.default_rng(seed)
    lens = np.repeat(rng.integers(0, 3 * PS, GROUPS), W)
    held = -(-lens // PS)
    order = rng.permutation(P).astype(np.int32)
    tables = np.full((B, MP), -1, np.int32)
    used = 0
    for r in range(B):
        tables[r, :held[r]] = order[used:used + held[r]]
        used += held[r]
    free = np.full(P, -1, np.int32)
    n = min(P - used, int(rng.integers(2, 12)))
    free[:n] = order[used:used + n]
    state = np.concatenate([lens, held, [n]]).astype(np.int32)
    new = np.repeat(rng.integers(0, 7, GROUPS), W).astype(np.int32)
    new[rng.integers(0, GROUPS) * W:][:W] = -1
    return new, state, tables, tables.copy(), free


def without(new, status):
    """new_lens with nothing for the groups of which not all are granted."""
    bad = (status.reshape(-1, W) != 0).any(1)
    return np.where(np.repeat(bad, W), 0, new).astype(np.int32), bad


def live(o):
    """What the state counts: tables up to the length, owned pages, the stack."""
    s = o["state"]
    return ([o["tables"][r, :-(-s[r] // PS)].tolist() for r in range(B)],
            [o["owned"][r, :s[B + r]].tolist() for r in range(B)], o["free"][:s[2 * B]].tolist(),
            s.tolist())


def cases():
    """Seeds whose first map refuses some beams of a group and grants others."""
    found = []
    for seed in range(200):
        new, state, *pool = start(seed)
        o = ref.kv_map(PS, P, 64, new, state, *pool)
        part = (o["status"].reshape(-1, W) != 0)
        if (part.any(1) & ~part.all(1)).any():
            found.append(seed)
    return found


def test_a_step_can_be_mapped_again():
    seeds = cases()
    assert len(seeds) > 20
    for seed in seeds:
        new, state, *pool = start(seed)
        first = ref.kv_map(PS, P, 64, new, state, *pool)
        again, bad = without(new, first["status"])
        assert bad.any()
        got = ref.kv_map(PS, P, 64, again, state, first["tables"], first["owned"], first["free"])
        want = ref.kv_map(PS, P, 64, again, state, *pool)      # as if the first had not been
        assert live(got) == live(want)
        for n in ("starts", "slots", "positions", "rows", "status"):
            assert np.array_equal(got[n], want[n]), n
        assert (got["status"] == 0).all()
        pages = sum(live(got)[1], []) + live(got)[2]
        assert len(set(pages)) == len(pages)


@pytest.mark.gpu
def test_a_step_can_be_mapped_again_on_the_gpu():
    """The same calls on the device, the second's new_lens worked out there."""
    import torch
    from ternary_weight_decoder_amd import binding as tb
    for seed in cases()[:12]:
        print(f"[map again] seed {seed}", flush=True)
        new, state, *pool = start(seed)
        first = ref.kv_map(PS, P, 64, new, state, *pool)
        again, _ = without(new, first["status"])
        want = ref.kv_map(PS, P, 64, again, state, first["tables"], first["owned"], first["free"])
        t, o, f, s, n = (torch.from_numpy(a.copy()).cuda() for a in (*pool, state, new))
        p = tb.KvPool(P, PS, t, o, f)
        i32 = dict(dtype=torch.int32, device="cuda:0")
        out = {k: torch.empty(c, **i32) for k, c in (
            ("state", 2 * B + 1), ("starts", B + 1), ("slots", 64), ("positions", 64), ("rows", 64),
            ("status", B))}
        tb.bitnet_kv_map_into(p, 64, n, s, *out.values())
        refused = (out["status"].view(-1, W) != 0).any(1).repeat_interleave(W)
        tb.bitnet_kv_map_into(p, 64, n.masked_fill(refused, 0), s, *out.values())
        assert np.array_equal(s.cpu().numpy(), state)
        out.update(tables=t, owned=o, free=f)
        for k, w in want.items():
            assert np.array_equal(out[k].cpu().numpy(), w), k
