"""Limits of the cache and answer calls that the host alone decides: no GPU needed."""

import pytest

import verify_draft_prep_gb300 as sd


@pytest.fixture(scope="module")
def lib():
    sd.build()
    return sd.load()


@pytest.mark.parametrize("D", [16, 64, 80, 128])
def test_attend_scratch_has_room_to_be_aligned(lib, D):
    """The parts are written 32 bytes at a time and take a whole number of them; a caller's scratch
    begins at any multiple of 16, so there are 16 bytes more than the parts take."""
    assert lib.sd_kv_attend_workspace_bytes(D) % 32 == 16


P = 256  # a well aligned dummy address; no call below gets as far as using it
END = 2 ** 31 - 1
CACHE = [P, P, 2048, 128, 64, P, P, 4, 16]  # k, v, strides, scales, num_blocks, block_size


def write(lib, n):
    return lib.sd_kv_write(n, 2, 64, P, 128, 64, P, 128, 64, P, *CACHE, None, None)


def read(lib, n):
    return lib.sd_kv_read(2, n, 2, 64, *CACHE, P, 4, P, None, P, P, 128, 64, None, None)


def attend(lib, B, n, Hq, Hkv):
    return lib.sd_kv_attend(B, n, 8, Hq, Hkv, 64, P, 256, 64, *CACHE, P, 4, P, P, 0.125, 1, P, 256,
                            64, None, P, 1 << 40, None, None)


@pytest.mark.parametrize("below", [0, 1, 15, 255, 1022])
def test_counts_near_the_end_of_int_are_refused(lib, below):
    """The kernels step over tokens and rows in int: within a step of its end they would wrap around
    and, over rows, never end."""
    n = END - below
    assert write(lib, n) == -2
    assert read(lib, n) == -2
    assert attend(lib, 2, n, 1, 1) == -2
    assert attend(lib, n, 3, 4, 2) == -2


def test_rows_of_shared_heads_count_too(lib):
    assert attend(lib, 2, END // 16, 16, 1) == -2
    assert attend(lib, 2, END // 48, 48, 2) == -2


def test_heads_that_one_token_cannot_have_are_refused(lib):
    """A CTA counts a token's heads times its tokens in int."""
    for Hkv in (END, 1 << 30, (1 << 22) + 1):
        assert lib.sd_kv_write(3, Hkv, 64, P, 128, 64, P, 128, 64, P, *CACHE, None, None) == -2
        assert lib.sd_kv_read(2, 3, Hkv, 64, *CACHE, P, 4, P, None, P, P, 128, 64, None, None) == -2
        assert lib.sd_kv_attend(2, 3, 8, Hkv, Hkv, 64, P, 256, 64, *CACHE, P, 4, P, P, 0.125, 1, P,
                                256, 64, None, P, 1 << 40, None, None) == -2


def test_calls_at_the_same_time_do_not_share_scratch(monkeypatch):
    """Two threads inside sd_kv_attend, neither with a workspace of its own."""
    import threading

    import torch

    inside, seen = threading.Barrier(2, timeout=60), []

    class Fake:
        @staticmethod
        def sd_kv_attend_workspace_bytes(D):
            return 4096

        @staticmethod
        def sd_kv_attend(*args):
            ws, size = args[-4:-2]
            seen.append((ws, size))
            inside.wait()
            return 0

    monkeypatch.setattr(sd, "_lib", Fake)
    monkeypatch.setattr(sd, "_attend_bytes", {}, raising=False)
    monkeypatch.setattr(sd, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(sd, "_raw_stream", lambda t, stream: 0)
    monkeypatch.setattr(sd, "_device", lambda t: t.device)
    c = torch.zeros(2, 4, 16, 2, 64, dtype=torch.uint8)
    s = torch.zeros(4, 2)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    table, lens, cu = (torch.zeros(n, dtype=torch.int32) for n in ((1, 4), (1,), (2,)))

    def call():
        sd.sd_kv_attend(q, c[0], c[1], s, s, table, lens, cu, torch.zeros_like(q))

    threads = [threading.Thread(target=call) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    (a, size), (b, _) = seen
    assert abs(a - b) >= size
