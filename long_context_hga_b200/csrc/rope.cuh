// Rotary positions with several axes, forward and backward.
//
// Pair p of a head's first rot_dim values turns by the angle
//   a = pos[axis[p]][token] * freq[p]:   (x, y) -> (x cos a - y sin a, y cos a + x sin a).
// The gradient of a rotation is the rotation by -a, so both directions are one
// kernel with a sign.  Pairs are (p, p + rot_dim/2) or, adjacent, (2p, 2p+1).
//
// Angles: freq is float64 and so is the product, from which whole turns are
// taken off before the rest goes to fp32, so a position of a million costs no
// accuracy.  A block computes the angles of its tokens once, in shared memory,
// and every head of q and k uses them.
//
// Bound: HBM (each value is read once and written once, 3 flops a value).  A
// thread moves one or two 16-byte vectors of each half at a time.  16384 tokens,
// 32 + 8 heads of 128, bf16: 63 us, 5.3 TB/s; the fp32 gradient of 4096: 31 us.
#pragma once
#include "common.cuh"

namespace hga {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxDim = 256;

struct RopeIo {
  const void* in;
  void* out;
  int64_t in_tok, in_head, out_tok, out_head;   // strides in elements
};

struct RopeArgs {
  const double* freq;       // [half]
  const uint8_t* axis;      // [half]
  const int32_t* pos;       // [n_axes][pos_stride] (stride 0: the same for all axes)
  int64_t pos_stride, n;
  int n_axes, half, d, adjacent;
  int heads0, heads;        // heads of io[0], heads of both
  int toks;                 // tokens per block
  float sign;
  RopeIo io[2];
};

template <typename T, int VEC>
struct RopeVec {
  static __device__ __forceinline__ void load(const T* p, float* f) {
    if constexpr (sizeof(T) == 2 && VEC == 8) {
      const uint4 r = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else if constexpr (sizeof(T) == 4 && VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        const float4 r = *reinterpret_cast<const float4*>(p + 4 * i);
        f[4 * i] = r.x; f[4 * i + 1] = r.y; f[4 * i + 2] = r.z; f[4 * i + 3] = r.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = Elt<T>::to_f32(p[i]);
    }
  }
  static __device__ __forceinline__ void store(T* p, const float* f) {
    if constexpr (sizeof(T) == 2 && VEC == 8) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (sizeof(T) == 4 && VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i)
        *reinterpret_cast<float4*>(p + 4 * i) =
            make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) p[i] = Elt<T>::from_f32(f[i]);
    }
  }
};

// VEC = 8 (16-byte vectors of bf16) needs 16-byte aligned rows and half % 8
// == 0, d % 8 == 0; VEC = 1 takes any layout.
template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  __shared__ float2 cs[8 * (kRopeMaxDim / 2)];
  griddep_wait();
  const int64_t t0 = (int64_t)blockIdx.x * a.toks;
  const int nt = (int)min((int64_t)a.toks, a.n - t0);
  for (int i = threadIdx.x; i < nt * a.half; i += kRopeThreads) {
    const int t = i / a.half, p = i - t * a.half;
    int ax = a.axis[p];
    if (ax >= a.n_axes) {
      report(HGA_ERR_DEVICE_CHECK);
      ax = 0;
    }
    const double turns = (double)a.pos[ax * a.pos_stride + t0 + t] * a.freq[p] *
                         0.15915494309189533577;   // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[t * a.half + p] = make_float2(c, a.sign * s);
  }
  __syncthreads();
  // Items of a head row: rotated vector pairs, then vectors past rot_dim.  A
  // thread keeps its item and goes from row to row, so that the index
  // arithmetic of a row is a few additions.
  const int rot_items = a.half / VEC, items = rot_items + (a.d - 2 * a.half) / VEC;
  const int rows = kRopeThreads / items;            // rows of a pass (items <= kRopeMaxDim)
  const int it = threadIdx.x % items;
  const int row = threadIdx.x / items;
  int t = row < rows ? row / a.heads : nt, hh = row % a.heads;   // past them: no row
  const int dt = rows / a.heads, dh = rows % a.heads;
#pragma unroll 2
  for (; t < nt; t += dt + (hh + dh >= a.heads), hh = hh + dh >= a.heads ? hh + dh - a.heads : hh + dh) {
    const RopeIo& io = a.io[hh >= a.heads0];
    const int h = hh >= a.heads0 ? hh - a.heads0 : hh;
    const TI* src = static_cast<const TI*>(io.in) + (t0 + t) * io.in_tok + h * io.in_head;
    TO* dst = static_cast<TO*>(io.out) + (t0 + t) * io.out_tok + h * io.out_head;
    float x[VEC], y[VEC];
    if (it >= rot_items) {
      const int at = 2 * a.half + (it - rot_items) * VEC;
      RopeVec<TI, VEC>::load(src + at, x);
      RopeVec<TO, VEC>::store(dst + at, x);
      continue;
    }
    const int ax = a.adjacent ? 2 * VEC * it : VEC * it;
    const int ay = a.adjacent ? ax + VEC : ax + a.half;
    RopeVec<TI, VEC>::load(src + ax, x);
    RopeVec<TI, VEC>::load(src + ay, y);
    const float2* c = cs + t * a.half + it * VEC;
    if (!a.adjacent || VEC == 1) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float u = x[j], v = y[j];
        x[j] = u * c[j].x - v * c[j].y;
        y[j] = v * c[j].x + u * c[j].y;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        float u = x[2 * j], v = x[2 * j + 1];
        x[2 * j] = u * c[j].x - v * c[j].y;
        x[2 * j + 1] = v * c[j].x + u * c[j].y;
        u = y[2 * j], v = y[2 * j + 1];
        const float2 e = c[VEC / 2 + j];
        y[2 * j] = u * e.x - v * e.y;
        y[2 * j + 1] = v * e.x + u * e.y;
      }
    }
    RopeVec<TO, VEC>::store(dst + ax, x);
    RopeVec<TO, VEC>::store(dst + ay, y);
  }
  // No griddep_launch: this kernel writes q, which a call with q_ready reads
  // without waiting, so its dependents start once all its blocks have ended.
}

}  // namespace hga
