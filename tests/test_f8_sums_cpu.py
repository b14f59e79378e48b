"""What the e4m3 products refuse of DMM_SHORT_SUMS, before any launch."""

import ctypes

import pytest

torch = pytest.importorskip("torch")
dmm = pytest.importorskip("decode_matmul_amd")
lib = dmm.raw()

DTYPE, ALIGN = 4, 5
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)      # never dereferenced


def test_short_sums_are_for_bf16():
    def dense(y, y_dtype, M=4):
        return lib.f8_matmul(FAKE, FAKE, M, 64, FAKE, FAKE, 16, None, y, y_dtype, None)

    def experts(y, y_dtype, M=4):
        return lib.f8_matmul_experts(FAKE, FAKE, M, 64, FAKE, FAKE, 16, 8, None, FAKE, FAKE, 2, y, y_dtype, None)

    for call in (dense, experts):
        for y_dtype in (dmm.TQ_F32 | 0x100, 2 | 0x100, 0x200 | 1, 0x300 | 1, -1):
            assert call(FAKE, y_dtype) == DTYPE
        assert call(ODD, dmm.TQ_BF16 | dmm.DMM_SHORT_SUMS) == ALIGN
        assert call(FAKE, dmm.TQ_BF16 | dmm.DMM_SHORT_SUMS, M=0) == 0
    # the other entry points take no such type
    assert lib.f8_unpack(FAKE, FAKE, 4, 64, 1, FAKE, dmm.TQ_BF16 | dmm.DMM_SHORT_SUMS, None, None) == DTYPE


def test_binding_refuses_short_sums_of_fp32():
    c, s = torch.zeros(2, 2, 128, dtype=torch.uint8), torch.zeros(2, 2)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: dmm.f8_matmul(c, s, 2, 200, c, s[:1], 2, torch.zeros(2, 2), short_sums=True),
                 lambda: dmm.f8_matmul_experts(c, s, 2, 200, c, s[:1], 2, torch.zeros(2, 2), 1, i, i, 1, short_sums=True)):
        with pytest.raises(TypeError):
            call()
