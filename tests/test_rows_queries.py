"""Workspace queries of the row-wise operators at the ends of their ranges, on the host."""
import ctypes
import subprocess
import sys

import pytest

import edge_message_passing_b200 as emp

P = 1 << 20            # a well aligned address that is never read


@pytest.mark.parametrize("dtype,y_dtype", [(0, 0), (1, 1), (2, 2), (3, 1)])
@pytest.mark.parametrize("fan_in,fan_out", [(64, 32), (2048, 2048), (2049, 1), (4096, 64), (65536, 65536)])
def test_zero_rows_need_no_workspace(fan_in, fan_out, dtype, y_dtype):
    """In a process of its own: a query that ends the process fails this test alone."""
    scale = P if dtype == 3 else None
    code = f"""if True:
        import ctypes, edge_message_passing_b200 as emp
        a = emp.DenseC(rows=0, fan_in={fan_in}, fan_out={fan_out}, dtype={dtype}, y_dtype={y_dtype}, x={P}, ldx={fan_in},
                       x_scale={scale}, weight={P}, ldw={fan_in}, w_scale={scale}, y={P}, ldy={fan_out})
        assert emp.lib().mp_dense_workspace_bytes(ctypes.byref(a)) == 0
        assert emp.lib().mp_dense(ctypes.byref(a), None, 0, None) == 0
    """
    run = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0, run.stderr[-500:]


@pytest.mark.parametrize("rows", [1, 16, 17, 129, 5000])
@pytest.mark.parametrize("fan_in,fan_out", [(1, 1), (2049, 3), (65536, 1), (1, 65536)])
def test_queries_of_all_sizes(rows, fan_in, fan_out):
    L = emp.lib()
    for dtype in (0, 1, 2):
        a = emp.DenseC(rows=rows, fan_in=fan_in, fan_out=fan_out, dtype=dtype, y_dtype=dtype, x=P, ldx=fan_in, weight=P, ldw=fan_in,
                       y=P, ldy=fan_out)
        g = emp.DenseGradC(rows=rows, fan_in=fan_in, fan_out=fan_out, dtype=dtype, g=P, ldg=fan_out, x=P, ldx=fan_in, weight=P,
                           ldw=fan_in, g_x=P, ldgx=fan_in, g_weight=P, g_bias=P)
        assert L.mp_dense_workspace_bytes(ctypes.byref(a)) % 256 == 0
        assert L.mp_dense_grad_workspace_bytes(ctypes.byref(g)) % 256 == 0
        g.rows = 0
        assert L.mp_dense_grad_workspace_bytes(ctypes.byref(g)) == 0
