"""CPU oracle (test infrastructure; never imported by the product path)."""
from .qgemv_oracle import (  # noqa: F401
    FP_FORMATS,
    abs_product_sum,
    e2m1_to_f64,
    e4m3_to_f64,
    e8m0_to_f64,
    fp_abs_product_sum,
    fp_dequantize,
    fp_elements,
    gather_abs_product_sum,
    qgemv_gather_reference,
    qgemv_fp_reference,
    bf16_bits_to_f64,
    check_close,
    dequantize,
    fp16_bits_to_f64,
    qgemv_add_reference,
    qgemv_reference,
    residual_f64,
    tolerance,
    unpack_codes,
)
from .kv_oracle import (  # noqa: F401
    append_places,
    attend_reference,
    round_e4m3,
    verify_reference,
    verify_weights,
    visible,
)
from .step_oracle import (  # noqa: F401
    adapt_reference,
    angle_reference,
    rotate_reference,
    route_reference,
)
