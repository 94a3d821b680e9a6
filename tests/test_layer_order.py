"""The rows of the gains' gradients, which the declared order fixes, are those that the library works with (CPU)."""
import random

import bitwise_reproducible_amd as br
import layer_order
import test_layer_host as host

KINDS = {"f32": 0, "bf16": 1}


def _sizes():
    yield 1024, [64, 8], 128, 128, 0, "bf16"  # 769 rows: one more than 768, each side rounded up for itself
    rng = random.Random(3)
    for _ in range(600):
        dim = 2 * rng.choice([rng.randint(1, 16), rng.randint(1, 256), 32, 64])
        yield (int(2 ** rng.uniform(0, 18)), [rng.randint(0, 64), rng.randint(0, 16)], dim,
               2 * rng.randint(1, dim // 2), rng.randint(0, 1), rng.choice(["f32", "bf16"]))


def test_workspace_holds_the_declared_rows():
    lib = br.layer._lib()
    for tokens, heads, dim, rotary, interleaved, kind in _sizes():
        _, rows = layer_order.rows_of(tokens, heads, dim, rotary, interleaved, kind)
        for given in ((0,), (1,), (0, 1)):
            a = host._args(batch=1, seq=tokens, dim=dim, rotary=rotary, dtype=KINDS[kind], interleaved=interleaved)
            for i in range(2):
                a.heads[i] = heads[i]
                a.gain[i] = host.P if i in given else None
            want = sum(-(-rows[i] * dim * 4 // 16) * 16 for i in given)
            assert lib.repro_qk_workspace_bytes(bytes(a)) == want, (tokens, heads, dim, rotary, kind, given)


def test_rows_round_up_for_each_side():
    assert sum(layer_order.rows_of(1024, [64, 8], 128, 128, 0, "bf16")[1]) == 769
    assert sum(layer_order.rows_of(16384, [16, 4], 128, 128, 0, "bf16")[1]) <= 768


def test_sizes_up_to_the_declared_limit_are_taken():
    lib = br.layer._lib()
    rng = random.Random(5)
    for _ in range(400):
        dim = 2 * rng.randint(1, 256)
        rotary, interleaved, kind = 2 * rng.randint(1, dim // 2), rng.randint(0, 1), rng.choice(["f32", "bf16"])
        padded = layer_order.padded_groups(dim, rotary, interleaved, kind)
        most = (2 ** 32 - 512) // padded  # heads in all, over the tokens
        both = int(2 ** rng.uniform(0.5, 20))
        tokens = min(most // both, 2 ** 31 - 1)
        heads = rng.randint(0, both)
        a = host._args(batch=1, seq=tokens, dim=dim, rotary=rotary, dtype=KINDS[kind], interleaved=interleaved)
        a.heads[:] = [heads, both - heads]
        for gain in (None, host.P):
            a.gain[0] = gain
            assert lib.repro_qk_workspace_bytes(bytes(a)) >= 0, (tokens, both, dim, rotary, kind)
        a.seq = 2 ** 31
        assert lib.repro_qk_workspace_bytes(bytes(a)) == -1
