"""Calls of the grouped and 4-bit products at the ends of the documented sizes
on the CPU (tests/experts_dry_run.py), their host code built so that a signed
overflow ends the process.  Prints each call ahead of it."""
import subprocess
import sys
import types

from dense_gemm_row_amd import gemm, w4
from tests import experts_dry_run

TOP = 2 ** 31 - 1
FAR = [TOP, TOP - 7, TOP - 15, TOP - 62, TOP - 126, TOP - 254, TOP - 255, 2 ** 30 + 1]
F32, BF16 = gemm.DTYPE_F32, gemm.DTYPE_BF16
O, X, W, Y, Q, S, Z = (i << 52 for i in range(1, 8))  # never dereferenced


def run(cmd, **kw):
    trap = [flag for f in ("-fsanitize=signed-integer-overflow", "-fsanitize-trap=signed-integer-overflow")
            for flag in ("-Xarch_host", f)]
    if "-fwrapv" in cmd:
        at = cmd.index("-fwrapv")
        cmd = cmd[:at] + trap + cmd[at + 1:]
    return subprocess.run(cmd, **kw)


def calls():
    for far in FAR:
        for T, K, N, G in ((far, 8, 8, 1), (far, 8, 8, 65535), (3, 8, far, 2), (3, far, 8, 2), (1, far, 16, 4000)):
            for dtype in (F32, BF16):
                for trans in (0, 1):
                    ldw = K if trans else N
                    yield ("gemm_grouped_matmul", dtype, dtype, trans, G, T, N, K, O, X, K, W, ldw, (N if trans else K) * ldw, Y, N, 1,
                           None)
                yield ("gemm_grouped_wgrad", dtype, F32, G, T, K, N, O, X, K, Y, N, W, N, K * N, 1.0, 0.0, None)
        for N, K in ((far, 32), (far, 300), (3, min(far, 2 ** 30))):
            for group in w4.GROUPS:
                ng, ldq = -(-K // group), -(-K // 32) * 16
                q = w4.GemmW4(Q, ldq, N * ldq, S, ng, N * ng, Z, ng, N * ng, group)
                for M in (1, 40, 128):
                    yield "gemm_w4_matmul", BF16, M, N, K, X, K, q, Y, N, None, 0, None
                yield "gemm_w4_grouped", BF16, 2, 2, N, K, O, X, K, q, Y, N, 1, None, 0, None
                for trans in (0, 1):
                    yield "gemm_w4_quantize", BF16, BF16, trans, N, K, X, N if trans else K, q, None
                yield "gemm_w4_dequantize", F32, BF16, N, K, q, X, K, None


def main(folder):
    experts_dry_run.subprocess = types.SimpleNamespace(run=run)
    dry = experts_dry_run.compile_dry(folder)
    for name, *args in calls():
        print(name, [a.group if isinstance(a, w4.GemmW4) else a for a in args], flush=True)
        status, _ = dry(name, *args)
        assert status == gemm.GEMM_OK, status
    print("every call returned")


if __name__ == "__main__":
    main(sys.argv[1])
