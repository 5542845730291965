"""CPU check: a product whose result starts where an operand does is refused; other work groups still read what one has written."""
import ctypes

import adam_ob_compress_amd as ob


def test_result_in_an_operands_place_is_refused():
    lib = ob.lib()

    def status(**kw):
        p = ob.ob_product(batch=1, m=64, n=64, k=64, a=0x10000, a_row=64, a_col=1, b=0x20000, b_row=64, b_col=1, c=0x30000, c_row=64,
                          d=0x40000, d_row=64, in_type=1, out_type=1, alpha=1.0)
        for k, v in kw.items():
            setattr(p, k, v)
        return lib.ob_matmul(ctypes.byref(p), None)

    assert status(d=0x10000) == 1 and status(d=0x20000) == 1
    assert status(d=0x10000, beta=1.0, c=0x10000) == 1
    assert status(d=0x10000, batch=0) == 0 and status(d=0x10000, m=0) == 0   # nothing to write
