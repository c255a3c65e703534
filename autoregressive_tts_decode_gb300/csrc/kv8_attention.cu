// kv8_attention.cu -- attention of new rows over the 8-bit cache.
//
// For row i of a sequence and head h of kv head g, with p over the positions it sees,
//   s_p = 2^(a_p) q . c_p / sqrt(hd),  o = sum_p e^(s_p - m) 2^(b_p) d_p / sum_p e^(s_p - m),
// c_p and d_p the codes of key and value, 2^(a_p) and 2^(b_p) their blocks' powers, m the
// largest score so far; o = 0 when it sees none.  A warp has one row of one head
// and goes through its positions one by one.
#include "kv8.cuh"

namespace q3 {

namespace {

constexpr int KA_THREADS = 128;

template <class T, int HD>
__global__ void __launch_bounds__(KA_THREADS) kv8_rows_kernel(const __grid_constant__ Kv8AttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int EPL = HD / 32;  // elements of a lane
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y, seq = blockIdx.z, i = blockIdx.x * (KA_THREADS / 32) + (threadIdx.x >> 5);
  Kv8Seq t;
  if (!kv8_seq(a.r, a.c.page, seq, true, t) || i >= t.n) return;
  const int row = t.row0 + i, g = h / (a.Hq / a.c.Hkv);
  const T* qp = static_cast<const T*>(a.q) + (size_t)row * a.ldq + h * HD + lane * EPL;
  float q[EPL], o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) {
    q[e] = to_f(qp[e]) / sqrtf((float)HD);
    o[e] = 0.f;
  }
  const unsigned long long mask = a.masks ? a.masks[row] : 0;
  const int end = t.L + (a.masks ? t.n : i + 1);
  float m = -INFINITY, l = 0.f;
  for (int p = 0; p < end; ++p) {
    if (p >= t.L && a.masks && !((mask >> (p - t.L)) & 1)) continue;
    int page = __ldg(a.r.page_table + (size_t)seq * a.r.pps + p / a.c.page);
    if (page < 0 || page >= a.c.n_pages) {
      op_status(a.r.status, Q3TTS_ERR_ARG);
      page = 0;
    }
    const long long kr = kv8_row(a.c, page, 0, g, p % a.c.page), vr = kv8_row(a.c, page, 1, g, p % a.c.page);
    float f[4];
    auto load = [&](long long at) {
      const uint8_t* c = a.c.codes + at * HD + lane * EPL;
      fp8x4_to_f32(EPL == 4 ? *reinterpret_cast<const uint32_t*>(c) : *reinterpret_cast<const uint16_t*>(c), f);
    };
    load(kr);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < EPL; ++e) s = fmaf(q[e], f[e], s);
    s = warp_sum(s) * kv8_power(a.c.powers[kr / a.c.block]);
    load(vr);
    const float top = fmaxf(m, s), was = expf(m - top), w = expf(s - top);
    const float wv = w * kv8_power(a.c.powers[vr / a.c.block]);
    m = top;
    l = l * was + w;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = fmaf(wv, f[e], o[e] * was);
  }
  T* op = static_cast<T*>(a.out) + (size_t)row * a.ldo + h * HD + lane * EPL;
#pragma unroll
  for (int e = 0; e < EPL; ++e) op[e] = from_f<T>(l > 0.f ? o[e] / l : 0.f);
}

}  // namespace

int launch_kv8_attention(const Kv8AttnArgs& a, int layers, int dtype, cudaStream_t s) {
  const dim3 grid((a.r.max_rows + 3) / 4, a.Hq, a.r.n_seqs);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, dim3(KA_THREADS), 0, s, a) == cudaSuccess ? Q3TTS_OK : Q3TTS_ERR_CUDA;
  };
  if (dtype == Q3TTS_F32) return a.c.hd == 128 ? go(kv8_rows_kernel<float, 128>) : go(kv8_rows_kernel<float, 64>);
  return a.c.hd == 128 ? go(kv8_rows_kernel<bf16, 128>) : go(kv8_rows_kernel<bf16, 64>);
}

}  // namespace q3
