// delta_step.hip -- the gated delta rule token by token (gfx950): the serving form (one token of each request on a
// pool of states) and the forward of very short rows.
//
//     S <- a S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q
//
// Bound by the states: 2 x 4 dk dv bytes a token and head against 7 dk dv operations.  A workgroup takes one
// (row, head) and 64 columns of its state, held in registers from the load to the store: 16 row groups x 16 lanes
// of 4 columns, so a state row is read as whole 256-byte runs and every load is in flight at once.  With
// o = scale (S^T q + (k.q) u) taken on the decayed state before its update, S^T k and S^T q share one reduction
// over the row groups (two lane exchanges, one pass through LDS, one barrier a token).  256 requests x 16 heads of
// 128 x 128: 106 us for 540 MB, 5.1 TB/s; one request of 5 heads of 64 x 64: 5 us on the card, 9.6 us with the call.
#include "sfm_delta.h"
#include "sfm_device.h"

namespace sfm {

namespace {

constexpr int kCols = 64;    // columns to a workgroup
constexpr int kGroups = 16;  // row groups
typedef float vec4 __attribute__((ext_vector_type(4)));

template <typename T, int RPT, bool VEC, bool STREAM>
__global__ __launch_bounds__(256) void delta_recurrent_kernel(const DeltaParams p, unsigned tiles) {
    __shared__ float red[2][2][4][kCols];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const unsigned unit = blockIdx.x / tiles;
    const int c0 = (int)(blockIdx.x - unit * tiles) * kCols + (tid & 15) * 4;
    const int s = (int)(unit / (unsigned)p.H), h = (int)(unit - (unsigned)s * p.H);
    const int rg = tid >> 4;
    int64_t first;
    int len;
    delta_row(p, s, first, len);
    int64_t slot = s;
    if (p.slots) {
        slot = p.slots[s];
        if (slot < 0 || slot >= p.pool) slot = -1;
    }
    const int64_t sbase = (slot * p.H + h) * (int64_t)p.dk * p.dv;
    const int hk = (int)((unsigned)h / (unsigned)p.share);
    const bool full = VEC && c0 + 4 <= p.dv;

    float S[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + kGroups * i;
#pragma unroll
        for (int c = 0; c < 4; ++c) S[i][c] = 0.0f;
        if (p.h0 && slot >= 0 && r < p.dk) {
            const float* sp = p.h0 + sbase + (int64_t)r * p.dv + c0;
            if (full) {
                const vec4* v = reinterpret_cast<const vec4*>(sp);
                const vec4 x = STREAM ? __builtin_nontemporal_load(v) : *v;
#pragma unroll
                for (int c = 0; c < 4; ++c) S[i][c] = x[c];
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c0 + c < p.dv) S[i][c] = sp[c];
            }
        }
    }

    for (int t = 0; t < len; ++t) {
        const int64_t tok = first + t;
        const T* qp = static_cast<const T*>(p.q) + tok * p.ldq + (int64_t)hk * p.dk;
        const T* kp = static_cast<const T*>(p.k) + tok * p.ldk + (int64_t)hk * p.dk;
        const T* vp = static_cast<const T*>(p.v) + tok * p.ldv + (int64_t)h * p.dv;
        // every wave takes the whole q and k (two elements a lane) and their norms and product for itself
        float q0 = 0.0f, q1 = 0.0f, k0 = 0.0f, k1 = 0.0f;
        if (lane < p.dk) q0 = to_f32(qp[lane]), k0 = to_f32(kp[lane]);
        if (RPT > 4 && lane + 64 < p.dk) q1 = to_f32(qp[lane + 64]), k1 = to_f32(kp[lane + 64]);
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = c0 + c < p.dv ? to_f32(vp[c0 + c]) : 0.0f;
        float g = to_f32(static_cast<const T*>(p.g)[tok * p.H + h]);
        const float beta = to_f32(static_cast<const T*>(p.beta)[tok * p.H + h]);
        g = g < kDeltaMinGate ? kDeltaMinGate : g;
        const float a = exp2_fast(g * kLog2e);
        float qq = q0 * q0 + q1 * q1, kk = k0 * k0 + k1 * k1, kq = k0 * q0 + k1 * q1;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            qq += __shfl_xor(qq, m);
            kk += __shfl_xor(kk, m);
            kq += __shfl_xor(kq, m);
        }
        float rq = p.scale, rk = 1.0f;
        if (p.l2norm) {
            rq *= 1.0f / __builtin_sqrtf(qq + kDeltaNormEps);
            rk = 1.0f / __builtin_sqrtf(kk + kDeltaNormEps);
        }
        q0 *= rq, q1 *= rq, k0 *= rk, k1 *= rk;
        kq *= rq * rk;

        float kr[RPT], sk[4] = {0, 0, 0, 0}, sq[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const int r = rg + kGroups * i;  // rows past dk hold zeros
            kr[i] = __shfl(i < 4 ? k0 : k1, r & 63);
            const float qr = __shfl(i < 4 ? q0 : q1, r & 63);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                S[i][c] *= a;
                sk[c] = __builtin_fmaf(kr[i], S[i][c], sk[c]);
                sq[c] = __builtin_fmaf(qr, S[i][c], sq[c]);
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            sk[c] += __shfl_xor(sk[c], 16);
            sq[c] += __shfl_xor(sq[c], 16);
            sk[c] += __shfl_xor(sk[c], 32);
            sq[c] += __shfl_xor(sq[c], 32);
        }
        float(*rd)[4][kCols] = red[t & 1];  // two buffers: one barrier a token
        if (lane < 16) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                rd[0][wave][lane * 4 + c] = sk[c];
                rd[1][wave][lane * 4 + c] = sq[c];
            }
        }
        __syncthreads();
        float u[4];
        const int cl = (tid & 15) * 4;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float x = (rd[0][0][cl + c] + rd[0][1][cl + c]) + (rd[0][2][cl + c] + rd[0][3][cl + c]);
            u[c] = beta * (v[c] - x);
        }
        if (rg == 0) {
            T* op = static_cast<T*>(p.o) + (tok * p.H + h) * (int64_t)p.dv + c0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float x = (rd[1][0][cl + c] + rd[1][1][cl + c]) + (rd[1][2][cl + c] + rd[1][3][cl + c]);
                if (c0 + c < p.dv) op[c] = from_f32<T>(slot < 0 ? 0.0f : __builtin_fmaf(kq, u[c], x));
            }
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) S[i][c] = __builtin_fmaf(kr[i], u[c], S[i][c]);
    }

    if (!p.hT || slot < 0) return;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
        const int r = rg + kGroups * i;
        if (r >= p.dk) continue;
        float* sp = p.hT + sbase + (int64_t)r * p.dv + c0;
        if (full) {
            const vec4 x = {S[i][0], S[i][1], S[i][2], S[i][3]};
            vec4* v = reinterpret_cast<vec4*>(sp);
            if (STREAM)
                __builtin_nontemporal_store(x, v);
            else
                *v = x;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (c0 + c < p.dv) sp[c] = S[i][c];
        }
    }
}

template <typename T, int RPT>
hipError_t launch_rpt(const DeltaParams& p, hipStream_t s) {
    const unsigned tiles = (p.dv + kCols - 1) / kCols;
    const dim3 grid((unsigned)p.rows * p.H * tiles);
    // States that outgrow the dies' L2 caches (32 MB together) pass them by: 107 us for 537 MB of them, 131 us without;
    // smaller ones stay for the next step.
    const bool stream = (int64_t)p.rows * p.H * p.dk * p.dv * 4 > 32 << 20;
    if (p.vec_s && stream)
        hipLaunchKernelGGL((delta_recurrent_kernel<T, RPT, true, true>), grid, dim3(256), 0, s, p, tiles);
    else if (p.vec_s)
        hipLaunchKernelGGL((delta_recurrent_kernel<T, RPT, true, false>), grid, dim3(256), 0, s, p, tiles);
    else
        hipLaunchKernelGGL((delta_recurrent_kernel<T, RPT, false, false>), grid, dim3(256), 0, s, p, tiles);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const DeltaParams& p, hipStream_t s) {
    if (p.dk <= 32) return launch_rpt<T, 2>(p, s);
    if (p.dk <= 64) return launch_rpt<T, 4>(p, s);
    return launch_rpt<T, 8>(p, s);
}

}  // namespace

hipError_t launch_delta_recurrent(const DeltaParams& p, int io_dtype, hipStream_t s) {
    return io_dtype == 0 ? launch_t<float>(p, s) : launch_t<__bf16>(p, s);
}

}  // namespace sfm
