"""GPU parity of matrices in 8 bits: written (bit for bit the format's), read
back and multiplied, against the fp64 oracle.

Products of codes are exact. Where all codes are small whole numbers and the
scales powers of two near one, every partial sum is exact in fp32 too, so
results have to be the oracle's, rounded once. Otherwise, with A = sum |a w| and
u = 2^-24: the matrix units take 32 products at a time into a sum that they cut
off, 2 u A for each step of 32 and up to 32 steps before the sum moves on; the
sums are then added, K / 1024 + 16 of them at u A: (64 + 16 + K / 1024 + 4) u A,
plus the rounding."""
import numpy as np
import pytest

from layer_helpers import HALF, U, done, eight, empty, host, own_status, tdtype, untouched, upload, upload_eight
from oracle import layer_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    import torch
    from nystr_self_attention_gb300 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    torch.cuda.set_device(0)
    import nystr_self_attention_gb300 as N
    own_status(N)


def values(rows, K, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(rows, K)) * 10.0 ** rng.uniform(-3, 3, (rows, 1)) * (1 + 20 * (rng.random(K) > 0.97))
    x[rng.random(x.shape) < 0.05] = 0.0
    return R.rounded(x, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", [(1, 16), (8, 128), (3, 144), (40, 512), (128, 528), (136, 1040), (264, 2064)])
def test_write_and_read(rows, K, block_rows, turned, dtype):
    import nystr_self_attention_gb300 as N
    if turned and rows % 8:
        rows += 8 - rows % 8
    x = values(rows, K, dtype, rows + K)
    codes, bytes_ = R.q8_write(x, block_rows)
    q = eight(N, rows, K, 32)
    N.nystrom_q8_write(q, upload(x.T, dtype, 8).T if turned else upload(x, dtype, 8), block_rows)
    done(N)
    assert (q.scales.cpu().numpy() == R.q8_words(bytes_)).all()
    got = q.codes.cpu().numpy()
    # the code of zero keeps a sign that the oracle may not
    assert (np.where(got == 128, 0, got) == np.where(codes == 128, 0, codes)).all()
    want = R.q8_read(codes, bytes_)
    for out_type in ("bf16", "f32"):  # 4 significant bits: exact in either
        out = empty(rows, K, out_type, 8)
        N.nystrom_q8_read(q, out)
        done(N)
        assert (host(out) == want).all() and untouched(out, K)


def test_write_ties_and_borders():
    """Halfway between codes, just beside it, subnormal codes, the largest of a
    block at 448, 449 and 480 times a power of two."""
    import nystr_self_attention_gb300 as N
    mags = R.VALUES[:127]
    mid = (mags[1:] + mags[:-1]) / 2
    x = np.zeros((12, 128), np.float64)
    x[0, :126], x[1, :126] = mid, -mid
    x[2, :126], x[3, :126] = np.nextafter(mid.astype(np.float32), np.float32(np.inf)), np.nextafter(mid.astype(np.float32), np.float32(0))
    x[:4, 127] = 448
    x[4, :3], x[5, :3], x[6, :3] = (448, 1, 2), (449, 1, 2), (480, 1, 2)
    x[7, 0], x[8, 0] = 448 * 2.0 ** -140, 2.0 ** -149
    x[9, :2] = 3.3e38, 1.0
    x[10, 5], x[11, 5] = np.inf, np.nan
    codes, bytes_ = R.q8_write(x)
    q = eight(N, 12, 128)
    N.nystrom_q8_write(q, upload(x, "f32"))
    done(N)
    got, words = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    assert (words == R.q8_words(bytes_)).all()
    assert (got[:10] == np.where(codes[:10] == 128, 0, codes[:10])).all() or (got[:10] & 127 == codes[:10] & 127).all()
    out = empty(12, 128, "f32")
    N.nystrom_q8_read(q, out)
    done(N)
    assert np.isnan(host(out)[10:]).all() and not np.isnan(host(out)[:10]).any()


def whole(rows, K, seed, spread=2):
    """Codes of whole numbers -4 .. 4 and scales of 2^-spread .. 2^spread."""
    rng = np.random.default_rng(seed)
    codes = R.e4m3_code(rng.integers(-4, 5, (rows, K)))
    return codes, (127 + rng.integers(-spread, spread + 1, (rows, -(-K // 128)))).astype(np.uint8)


MATMUL = [(1, 8, 16), (1, 128, 128), (2, 136, 528), (16, 1000, 1040), (17, 264, 4096), (32, 512, 2048), (33, 40, 8192),
          (64, 2000, 640), (65, 136, 144), (128, 1024, 1024), (129, 128, 512), (200, 264, 4112), (300, 1000, 656),
          (513, 2568, 1600), (1000, 136, 16384), (2049, 1160, 272)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,n,K", MATMUL)
def test_matmul_of_whole_numbers(T, n, K, dtype):
    """Sums below 16 * 16 * 4 * 16384 = 2^24 in steps of 2^-4: exact below 2^20 / 16;
    the largest here stay under 2^19."""
    import nystr_self_attention_gb300 as N
    a, ab = whole(T, K, T + K, 1)
    w, wb = whole(n, K, n + K, 1)
    want = R.q8_read(a, ab) @ R.q8_read(w, wb).T
    assert np.abs(R.q8_read(a, ab)).max() * np.abs(R.q8_read(w, wb)).max() * K < 2.0 ** 22
    out = empty(T, n, dtype, 8)
    N.nystrom_q8_matmul(upload_eight(N, a, R.q8_words(ab), 16), upload_eight(N, w, R.q8_words(wb), 48), out)
    done(N)
    assert (host(out) == R.rounded(want, dtype)).all()
    assert untouched(out, n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 16, 100, 300])
def test_matmul_of_any_codes(T, dtype):
    import nystr_self_attention_gb300 as N
    rng = np.random.default_rng(T)
    K, n = 2064, 520

    def some(rows):
        codes = rng.integers(0, 256, (rows, K)).astype(np.uint8)
        codes[(codes & 127) == 127] = 0x38
        return codes, (127 + rng.integers(-12, 13, (rows, -(-K // 128)))).astype(np.uint8)
    a, ab = some(T)
    w, wb = some(n)
    av, wv = R.q8_read(a, ab), R.q8_read(w, wb)
    want, A = av @ wv.T, np.abs(av) @ np.abs(wv).T
    out = empty(T, n, dtype)
    N.nystrom_q8_matmul(upload_eight(N, a, R.q8_words(ab)), upload_eight(N, w, R.q8_words(wb)), out)
    done(N)
    assert (np.abs(host(out) - want) <= (84 + K / 1024) * U * A + HALF[dtype] * np.abs(want)).all()


@pytest.mark.parametrize("T", [3, 200])
def test_matmul_keeps_nan_blocks_to_their_rows(T):
    import nystr_self_attention_gb300 as N
    a, ab = whole(T, 656, 1, 1)
    w, wb = whole(264, 656, 2, 1)
    ab[1, 5] = 255
    wb[130, 0] = 255
    out = empty(T, 264, "f32")
    N.nystrom_q8_matmul(upload_eight(N, a, R.q8_words(ab)), upload_eight(N, w, R.q8_words(wb)), out)
    done(N)
    bad = np.zeros((T, 264), bool)
    bad[1], bad[:, 130] = True, True
    assert (np.isnan(host(out)) == bad).all()


def test_refusals_in_python():
    import torch
    import nystr_self_attention_gb300 as N
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8, device="cuda"), torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        N.NystromQ8(codes.int(), scales)
    with pytest.raises(ValueError):
        N.NystromQ8(codes.T, scales)
    with pytest.raises(ValueError):
        N.NystromQ8(codes, scales[:, :2])
    with pytest.raises(N.NystromError):
        N.NystromQ8(codes[:, :24], scales)
    q = N.NystromQ8(codes, scales)
    with pytest.raises(ValueError):
        N.nystrom_q8_write(q, torch.zeros(4, 32, device="cuda"))
    with pytest.raises(ValueError):
        N.nystrom_q8_write(q, torch.zeros(4, 128, device="cuda")[:, ::2])
    with pytest.raises(N.NystromError):
        N.nystrom_q8_write(q, torch.zeros(4, 64, device="cuda"), block_rows=2)
    with pytest.raises(ValueError):
        N.nystrom_q8_read(q, torch.zeros(4, 32, device="cuda"))
    with pytest.raises(ValueError):
        N.nystrom_q8_matmul(q, q, torch.zeros(4, 8, device="cuda"))
    with pytest.raises(N.NystromError):
        N.nystrom_q8_matmul(q, q, torch.zeros(4, 4, device="cuda"))  # columns in eights


def test_write_ties_and_borders_with_their_signs():
    """The codes of test_write_ties_and_borders bit for bit, and those of negative
    zeros and of values that round to one."""
    import nystr_self_attention_gb300 as N
    mags = R.VALUES[:127]
    mid = (mags[1:] + mags[:-1]) / 2
    x = np.zeros((8, 128), np.float64)
    x[0, :126], x[1, :126] = mid, -mid
    above, below = (np.nextafter(mid.astype(np.float32), np.float32(v)) for v in (np.inf, 0))
    x[2, :126], x[3, :126], x[4, :126] = above, below, -below
    x[:5, 127] = 448
    x[5, ::2] = -0.0
    x[6, :3], x[7, :3] = (-448, -2.0 ** -10, 2.0 ** -10), (-3.3e38, -1.0, 1.0)
    for turned in (False, True):
        for block in (1, 128):
            codes, bytes_ = R.q8_write(x, block)
            q = eight(N, 8, 128)
            N.nystrom_q8_write(q, upload(x.T, "f32").T if turned else upload(x, "f32"), block)
            done(N)
            assert (q.scales.cpu().numpy() == R.q8_words(bytes_)).all()
            assert (q.codes.cpu().numpy() == codes).all()
