// The SiLU gate of the 8-bit products and of the few-token layer.
#pragma once

namespace moe {

// silu(g) * u for any g and u.  Past g = -87 the denominator 1 + e^-g leaves the
// range in which __fdividef divides (2^126; it gives 0 there), and past -89
// fp32, while a large u still makes the product a normal number.  From kGateFar
// on the sigmoid is e^g to fp32's last bit, taken as the square of its root with
// the second factor last, so that no step underflows before the product does.
constexpr float kGateFar = -80.0f;
__device__ __forceinline__ float silu_times_far(float g, float u) {
  const float t = expf(0.5f * g);
  return g * t * u * t;
}
// For g >= kGateFar (or NaN).  The division is good to 2 units and the
// exponential to 2 (ACCURATE) or to 2 + 1.16 |g|, which a result rounded to bf16
// does not show.
template <bool ACCURATE>
__device__ __forceinline__ float silu_times_near(float g, float u) {
  return __fdividef(g, 1.0f + (ACCURATE ? expf(-g) : __expf(-g))) * u;
}
template <bool ACCURATE>
__device__ __forceinline__ float silu_times_wide(float g, float u) {
  return g < kGateFar ? silu_times_far(g, u) : silu_times_near<ACCURATE>(g, u);
}

}  // namespace moe
