// Expert FFN with 8-bit integer weights (MOE_I8_CHANNEL): two products in
// 8-bit integers over the expert groups, each after a row quantisation.
//
//   q, s   = quantise(x)          per token row
//   h      = bf16(silu(g) u)      g, u = s (q W^T) w   (or relu)
//   q', s' = quantise(h)          per row
//   y      = bf16(s' (q' W3^T) w3)
//
// The intermediate is bf16, as with every other weight type; its row maximum
// spans all of the first product's output tiles, so it is quantised by a pass
// of its own (2 F bytes read, F written per row).  y is rounded to bf16 before
// the combine, as with every other weight type, because the staged calls hand
// it on in act_dtype: against 64 bits a top-8 layer's output is 2.3e-3 off, and
// 1.7e-3 (its own rounding alone) where moe_forward_few keeps y in fp32.
// Inside moe_forward the
// token rows are quantised once each and their codes written straight to the
// rows of their slots, which takes the place of the dispatch's row copy.
#include "common.cuh"

namespace moe {

cudaError_t launch_mm_i8(const MmI8Args &a, cudaStream_t s) {
  if (mm_i8_is_few(a)) return launch_mm_i8_few(a, s);
  static const int pairs = mm_i8_pairs();
  return pairs > 0 && mm_i8_is_large(a) ? launch_mm_i8_pair(a, pairs, s) : launch_mm_i8_tc(a, s);
}

cudaError_t launch_ffn_i8(const FfnArgs &a, cudaStream_t s) {
  const int32_t *present = a.offsets + a.E;
  cudaError_t err = a.slot_row
                        ? launch_quantize_rows(a.x, true, a.x_rows, a.d, a.q, a.qs, s, nullptr, a.slot_row, a.top_k)
                        : launch_quantize_rows(a.x, true, a.rows_cap, a.d, a.q, a.qs, s, present);
  if (err != cudaSuccess) return err;
  MmI8Args m{};
  m.offsets = a.offsets;
  m.G = a.E;
  m.rows_cap = a.rows_cap;
  m.N = a.F;
  m.K = a.d;
  m.b_stride = a.w_stride;
  m.mode = a.act == MOE_ACT_SWIGLU ? I8_SWIGLU : I8_RELU;
  m.q = a.q;
  m.xs = a.qs;
  m.w0 = static_cast<const int8_t *>(a.w1);
  m.w1 = static_cast<const int8_t *>(a.w2);
  m.ws0 = static_cast<const float *>(a.s1);
  m.ws1 = static_cast<const float *>(a.s2);
  m.out = a.h;
  m.status = a.status;
  if ((err = launch_mm_i8(m, s)) != cudaSuccess) return err;
  if (a.mid_event && (err = cudaEventRecord(a.mid_event, s)) != cudaSuccess) return err;
  // the first product is done with the codes of x: the codes of h take their place
  if ((err = launch_quantize_rows(a.h, true, a.rows_cap, a.F, a.q, a.qs, s, present)) != cudaSuccess) return err;
  m.N = a.d;
  m.K = a.F;
  m.b_stride = a.d;
  m.mode = I8_PLAIN;
  m.w0 = static_cast<const int8_t *>(a.w3);
  m.w1 = nullptr;
  m.ws0 = static_cast<const float *>(a.s3);
  m.ws1 = nullptr;
  m.out = a.y;
  return launch_mm_i8(m, s);
}

}  // namespace moe
