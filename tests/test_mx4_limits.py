"""The bound on rows and columns that ssd_mx4_quant documents holds for every
call on 4-bit operands: the size beyond is refused, the last one is not (by its
next check).  CPU only: no kernel is started."""
import pytest

from test_block_abi import BIG, DEQUANT, LINEAR, MATMUL, NULL, QUANT, UNSUPPORTED, call, mx4, put


@pytest.mark.parametrize("rows,columns", [(1 << 28, 512), (1 << 27, 1024), (1 << 20, 131072)])
@pytest.mark.parametrize("name,args,outputs,ws", [
    ("ssd_mx4_quant", QUANT, 0, None), ("ssd_mx4_dequant", DEQUANT, 0, None), ("ssd_mx4_matmul", MATMUL, 64, None),
    ("ssd_mx4_linear", LINEAR, 64, BIG)])
def test_rows_and_columns(name, args, outputs, ws, rows, columns):
    args = put(args, _0=None)
    assert call(name, mx4(rows=rows, columns=columns, outputs=outputs), *args, ws=ws) == UNSUPPORTED
    assert call(name, mx4(rows=rows - 16, columns=columns, outputs=outputs), *args, ws=ws) == NULL
