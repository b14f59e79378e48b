"""Which kernel an MXFP4 product runs, as launch_mx_matmul and launch_mx_gemm
decide it, and sizes that reach every one of them.

tests/test_mx_forms_cpu.py holds the rules here against the sources, so that a
changed threshold does not take a kernel's test away unnoticed;
tests/test_gpu_mx_forms.py runs the sizes.
"""

import itertools
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_matmul_amd", "csrc")
UNITS = 256                                     # compute units of the part


def _gemm(K, ldx, M, mx, grouped):
    return K * 2 < 1 << 24 and (mx or grouped or M == 1 or ldx * 2 < 1 << 24)


def dense_form(M, N, K, mx, ldx=0, aligned=True):
    """Template arguments of the kernel.  aligned: x (with mx, the scales) at 16 bytes."""
    tiles = lambda side: -(-M // side) * -(-N // side)
    direct = True if mx else aligned and (ldx % 8 == 0 or M == 1)
    rows, halves = -(-N // 16), -(-N // 32)
    few = 16 if not mx or 2 * halves <= UNITS or halves > 2 * UNITS else 8 if halves <= UNITS else 0
    if M > few and _gemm(K, ldx, M, mx, False):
        if tiles(32) <= 2 * UNITS:
            shape = (32, 32, 1, 1, 1 if mx else 4 if tiles(32) <= UNITS else 2, 4)
        elif 4 * tiles(256) >= 3 * UNITS:
            shape = (256, 256, 2, 4, 1 if mx else 2, 1)
        elif 4 * tiles(128) >= 3 * UNITS:
            shape = (128, 128, 2, 2, 1 if mx else 2, 1)
        else:
            shape = (64, 64, 2, 2, 2 if mx else 4, 1)
        if mx:
            direct = shape[0] == 64 and aligned and K % 512 == 0
        return ("gemm", mx, direct) + shape + (False,)
    if mx:
        shape = (16, 1, 8) if rows <= 2 * UNITS else (16, 2, 4)
    elif M <= 4:
        shape = (2 if M <= 2 else 4,) + ((1, 8) if rows <= 2 * UNITS else (2, 4))
    elif M <= 8:
        shape = (8,) + ((1, 8) if rows <= UNITS else (2, 8) if rows <= 2 * UNITS else (2, 4))
    else:
        shape = (16,) + ((1, 4) if rows <= UNITS else (2, 4) if rows <= 2 * UNITS else (4, 4))
    return ("gemv", mx) + shape + (direct, False)


def experts_form(M, top_k, E, K, ldx, aligned=True):
    direct = aligned and (ldx % 8 == 0 or M == 1)
    if M * top_k >= 6 * E and _gemm(K, ldx, M, False, True):
        shape = (32, 128, 1, 4, 4, 1) if M * top_k < 40 * E else (64, 256, 1, 4, 2, 1)
        return ("gemm", False, direct) + shape + (True,)
    return ("gemv", False, 8, 2, 4, direct, True)


def _body(file, function):
    """The function's body without comments, whitespace made one space."""
    text = open(os.path.join(CSRC, file)).read()
    text = text[text.index(function):]
    text = text[:text.index("\n}\n")]
    return re.sub(r"\s+", " ", re.sub(r"//[^\n]*", "", text))


def rules():
    """The text of everything that decides, in one string."""
    return "\n".join((_body("mx_gemv.hip", "hipError_t launch_mx_matmul("), _body("mx_gemm.hip", "bool mx_gemm_takes("),
                      _body("mx_gemm.hip", "hipError_t launch_mx_gemm("),
                      _body("mx_gemv.hip", "hipError_t launch_bf16("), _body("mx_gemm.hip", "hipError_t launch_bf16(")))


def forms_in_sources():
    """Template arguments of every kernel that the two functions can launch."""
    found = set()
    for kind, file, function in (("gemv", "mx_gemv.hip", "hipError_t launch_mx_matmul("),
                                 ("gemm", "mx_gemm.hip", "hipError_t launch_mx_gemm(")):
        for bf16, args in re.findall(r"launch(_bf16)?<([^>]*)>\(a, s\)", _body(file, function)):
            v = tuple(w == "true" if w in ("true", "false") else int(w) for w in re.split(r", *", args))
            if not bf16:
                found.add((kind,) + v)
                continue
            for direct in (True, False):
                found.add((kind, False, direct) + v if kind == "gemm" else (kind, False) + v[:3] + (direct, v[3]))
    return found


def _ld(K, direct):
    """A distance of rows for which x is (not) read in aligned pieces."""
    return -(-K // 8) * 8 + (0 if direct else 3)


# M, N, K, x in MXFP4, aligned.  K: several slabs or chunks (8999: two segments of scales)
# and a cut rest.  N: rows of y that are and that are not whole 16-byte pieces.
DENSE = []
for M, N in ((1, 70), (2, 301), (2, 8215), (3, 90), (4, 8216), (7, 4000), (5, 5001), (8, 8215), (13, 4000), (16, 8001),
             (9, 8216), (40, 4000)):
    DENSE += [(M, N, 8999, False, d) for d in (True, False)]
for M, N, K in ((64, 8000, 4101), (500, 4100, 1100), (497, 4104, 1535), (700, 4300, 1003), (1030, 12500, 1155)):
    DENSE += [(M, N, K, False, d) for d in (True, False)]
DENSE += [(1, 70, 8999, True, True), (5, 4000, 8999, True, True), (8, 8000, 4101, True, False),
          (13, 16401, 8999, True, True), (20, 4000, 4101, True, True), (16, 8001, 4097, True, False),
          (500, 4100, 1536, True, True), (500, 4100, 1536, True, False), (497, 4104, 1100, True, True),
          (700, 4300, 1155, True, True), (1030, 12500, 1155, True, False), (1030, 12500, 2048, True, True)]

# M, N, K, experts, top_k, rows' distance a multiple of 8, x at 16 bytes.  Few slots an expert,
# 6 to 39, and 40 or more; more experts than a workgroup has threads.
EXPERTS = [(M, N, K, 8, 2, d, a)
           for (M, N), K, (d, a) in itertools.product(((20, 150), (60, 300), (300, 520)), (1003, 331),
                                                      ((True, True), (False, True), (True, False)))]
EXPERTS += [(100, 40, 96, 512, 4, True, True), (1000, 40, 100, 300, 2, True, True), (3000, 40, 64, 300, 5, False, True),
            (1, 33, 4101, 4, 2, True, True), (7, 33, 9100, 2, 1, False, True)]

# M, N, K, experts: rows too long for the tiles, so that the streaming form takes several passes
LONG = [(20, 20, (1 << 23) + 40, False, 0), (20, 20, (1 << 23) + 40, True, 0), (20, 10, (1 << 23) + 40, False, 2)]


def dense_cases_form(M, N, K, mx, aligned):
    return dense_form(M, N, K, mx, _ld(K, aligned), aligned)


def experts_cases_form(M, N, K, E, top_k, direct, aligned):
    return experts_form(M, top_k, E, K, _ld(K, direct), aligned)
