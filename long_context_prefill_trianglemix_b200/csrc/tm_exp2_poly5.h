// Generated by gen_exp2_poly5.py; do not edit.
// 2^f ~ c0 + c1 f + ... + c5 f^5 on [-1/2, 1/2]: relative-error least squares on
// 2000 Chebyshev nodes; max relative error of the float32 coefficients 1.417e-07.
#pragma once
#define TM_EXP2_P5_C0 1.0000001192092896f
#define TM_EXP2_P5_C1 0.6931469440460205f
#define TM_EXP2_P5_C2 0.24022121727466583f
#define TM_EXP2_P5_C3 0.05550742521882057f
#define TM_EXP2_P5_C4 0.009675459936261177f
#define TM_EXP2_P5_C5 0.0013266970636323094f
