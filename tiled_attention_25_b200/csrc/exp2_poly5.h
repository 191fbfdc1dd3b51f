// Generated by gen_exp2_poly.py: minimax (relative error) polynomial for 2^f,
// f in [-0.5, 0.5], degree 5; max relative error 7.494e-08 (float64
// coefficients), 1.547e-07 with the float32 coefficients below.
#pragma once

namespace attn25 {

constexpr float kExp2E0 = 1.0000001192092896f;
constexpr float kExp2E1 = 0.6931469440460205f;
constexpr float kExp2E2 = 0.24022120237350464f;
constexpr float kExp2E3 = 0.05550713092088699f;
constexpr float kExp2E4 = 0.009675540961325169f;
constexpr float kExp2E5 = 0.0013276472454890609f;

}  // namespace attn25
