// gdn2_norm.hip -- layer norm and root-mean-square norm over the last axis,
// optionally times silu(gate), and their gradients.
//
//   c = x - mean(x) (layer) or x,  r = 1 / sqrt(mean(c^2) + eps),  xh = c r,
//   n = xh w + bias,  y = n silu(z)  (or n without a gate z).
// With dn = dy silu(z) and d = dn w:
//   dx = r (d - xh mean(d xh) - mean(d))   (the last term for layer norm only)
//   dw = sum over rows of dn xh,  dbias = sum over rows of dn,
//   dz = dy n silu'(z),  silu'(z) = s (1 + z (1 - s)),  s = sigmoid(z).
// The mean is taken first and the squares of the centred values second, so
// that a large common offset costs no accuracy. All sums are fp32.
#include "gdn2_device.hpp"
#include "gdn2_norm.hpp"

namespace gdn2 {

namespace {

constexpr int kNT = 256;

// Sum over the workgroup, the same value and rounding in every thread.
__device__ __forceinline__ float block_sum(float x, float *red, int tid) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) x += __shfl_xor(x, off, 64);
  __syncthreads();
  if ((tid & 63) == 0) red[tid >> 6] = x;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

__device__ __forceinline__ float load_w(const void *p, int i, bool bf16, float none) {
  if (!p) return none;
  return bf16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[i]) : static_cast<const float *>(p)[i];
}
__device__ __forceinline__ void store_w(void *p, int i, bool bf16, float v) {
  if (bf16)
    static_cast<uint16_t *>(p)[i] = f32_to_bf16(v);
  else
    static_cast<float *>(p)[i] = v;
}

// 1 / (1 + e^-z); z below -87 counts as -87 (2e-38), NaN stays.
__device__ __forceinline__ float sigmoid(float z) {
  z = z < -87.f ? -87.f : z;
  const float d = 1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f);
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r);
}

// A row's statistics, the row read from memory for each pass.
template <bool BF16>
__device__ __forceinline__ void loop_stats(const typename Elem<BF16>::T *x, const NormArgs &p, float *red, int tid,
                                           float &mean, float &r) {
  float s = 0.f;
  mean = 0.f;
  if (p.layer) {
    for (int c = tid; c < p.D; c += kNT) s += Elem<BF16>::ld(x + c);
    mean = block_sum(s, red, tid) / (float)p.D;
    s = 0.f;
  }
  for (int c = tid; c < p.D; c += kNT) {
    const float v = Elem<BF16>::ld(x + c) - mean;
    s = __builtin_fmaf(v, v, s);
  }
  r = 1.f / __builtin_sqrtf(block_sum(s, red, tid) / (float)p.D + p.eps);
}

// Any width and alignment: a workgroup a row, one value a thread at a time.
template <bool BF16, bool GATE>
__global__ __launch_bounds__(kNT) void norm_forward_loop(NormArgs p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  __shared__ float red[4];
  const int tid = threadIdx.x;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.x) + row * p.D;
    float mean, r;
    loop_stats<BF16>(x, p, red, tid, mean, r);
    for (int c = tid; c < p.D; c += kNT) {
      float y = (E::ld(x + c) - mean) * r * load_w(p.weight, c, p.wbf16, 1.f) + load_w(p.bias, c, p.wbf16, 0.f);
      if constexpr (GATE) {
        const float z = E::ld(static_cast<const T *>(p.gate) + row * p.D + c);
        y *= z * sigmoid(z);
      }
      E::st(static_cast<T *>(p.y) + row * p.D + c, y);
    }
  }
}

template <bool BF16, bool GATE>
__global__ __launch_bounds__(kNT) void norm_backward_loop(NormArgs p) {
  using E = Elem<BF16>;
  using T = typename E::T;
  __shared__ float red[4];
  const int tid = threadIdx.x;
  float *pw = static_cast<float *>(p.workspace) + (size_t)blockIdx.x * p.D;
  float *pb = static_cast<float *>(p.workspace) + ((size_t)gridDim.x + blockIdx.x) * p.D;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T *x = static_cast<const T *>(p.x) + row * p.D, *dy = static_cast<const T *>(p.dy) + row * p.D;
    const T *gate = static_cast<const T *>(p.gate) + row * p.D;
    float mean, r, sd = 0.f, sx = 0.f;
    loop_stats<BF16>(x, p, red, tid, mean, r);
    for (int c = tid; c < p.D; c += kNT) {
      const float xh = (E::ld(x + c) - mean) * r, w = load_w(p.weight, c, p.wbf16, 1.f);
      float dn = E::ld(dy + c);
      if constexpr (GATE) {
        const float z = E::ld(gate + c), s = sigmoid(z), n = xh * w + load_w(p.bias, c, p.wbf16, 0.f);
        if (p.dgate) E::st(static_cast<T *>(p.dgate) + row * p.D + c, dn * n * (s * (1.f + z * (1.f - s))));
        dn *= z * s;
      }
      if (p.dweight) pw[c] = row == blockIdx.x ? dn * xh : pw[c] + dn * xh;
      if (p.dbias) pb[c] = row == blockIdx.x ? dn : pb[c] + dn;
      sd += dn * w;
      sx += dn * w * xh;
    }
    sd = p.layer ? block_sum(sd, red, tid) / (float)p.D : 0.f;
    sx = block_sum(sx, red, tid) / (float)p.D;
    for (int c = tid; c < p.D; c += kNT) {
      const float xh = (E::ld(x + c) - mean) * r;
      float dn = E::ld(dy + c);
      if constexpr (GATE) {
        const float z = E::ld(gate + c);
        dn *= z * sigmoid(z);
      }
      E::st(static_cast<T *>(p.dx) + row * p.D + c, r * (dn * load_w(p.weight, c, p.wbf16, 1.f) - xh * sx - sd));
    }
  }
}

// Column sums of the partial sums, in a fixed order.
__global__ __launch_bounds__(kNT) void norm_reduce(NormArgs p, int parts) {
  __shared__ float red[16][17];
  const int tid = threadIdx.x, col = blockIdx.x * 16 + (tid & 15), grp = tid >> 4;
  void *out = blockIdx.y ? p.dbias : p.dweight;
  if (!out) return;
  const float *part = static_cast<const float *>(p.workspace) + (size_t)blockIdx.y * parts * p.D;
  float s = 0.f;
  if (col < p.D)
    for (int g = grp; g < parts; g += 16) s += part[(size_t)g * p.D + col];
  red[grp][tid & 15] = s;
  __syncthreads();
  if (tid < 16 && col < p.D) {
    s = 0.f;
#pragma unroll
    for (int g = 0; g < 16; ++g) s += red[g][tid];
    store_w(out, col, p.wbf16, s);
  }
}

int64_t parts_of(int64_t rows) { return rows < 1024 ? rows : 1024; }

}  // namespace

size_t norm_backward_workspace_bytes(int64_t rows, int D, bool bf16) {
  (void)bf16;
  return (size_t)parts_of(rows) * D * 2 * sizeof(float);
}

hipError_t launch_norm_forward(const NormArgs &p, hipStream_t st) {
  const dim3 grid((unsigned)(p.rows < 65536 ? p.rows : 65536));
  if (p.bf16)
    p.gate ? norm_forward_loop<true, true><<<grid, kNT, 0, st>>>(p) : norm_forward_loop<true, false><<<grid, kNT, 0, st>>>(p);
  else
    p.gate ? norm_forward_loop<false, true><<<grid, kNT, 0, st>>>(p) : norm_forward_loop<false, false><<<grid, kNT, 0, st>>>(p);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs &p, hipStream_t st) {
  const int parts = (int)parts_of(p.rows);
  const dim3 grid((unsigned)parts);
  if (parts == 0) {
    // no rows: the sums below are empty
  } else if (p.bf16)
    p.gate ? norm_backward_loop<true, true><<<grid, kNT, 0, st>>>(p) : norm_backward_loop<true, false><<<grid, kNT, 0, st>>>(p);
  else
    p.gate ? norm_backward_loop<false, true><<<grid, kNT, 0, st>>>(p) : norm_backward_loop<false, false><<<grid, kNT, 0, st>>>(p);
  if (p.dweight || p.dbias) norm_reduce<<<dim3((unsigned)((p.D + 15) / 16), 2), kNT, 0, st>>>(p, parts);
  return hipGetLastError();
}

}  // namespace gdn2
