// A mixture-of-experts layer for a few tokens (definition in sgemm.h): router, choice of
// experts, gated pair of 4-bit products and the 4-bit product back, summed over a token's
// experts.
#include "internal.cuh"
#include "q4.cuh"

namespace sgemm {
namespace {

constexpr int kMoeMaxT = 64;
constexpr int kMoeMaxDim = 16384;
constexpr int kMoeMaxE = 256;
constexpr int kMoeMaxTop = 16;

constexpr int WARPS = 8;

struct MoeArgs {
    const void* x;
    size_t ldx;
    const void* router;
    int router_dtype, dtype, T, D, F, E, top, renormalize;
    const uint8_t* live;
    int* ids;        // T x top, -1 for a token that is not live
    float* weights;  // T x top
    float* hidden;   // T x top x F
    void* y;
    size_t ldy;
};

__global__ void __launch_bounds__(WARPS * 32) moe_router_kernel(MoeArgs a) {
    __shared__ float logit[kMoeMaxE];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = blockIdx.x;
    for (int e = warp; e < a.E; e += WARPS) {
        float s = 0.0f;
        for (int d = lane; d < a.D; d += 32)
            s = fmaf(load_as_float(a.x, a.dtype, t * a.ldx + d),
                     load_as_float(a.router, a.router_dtype, size_t(e) * a.D + d), s);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) logit[e] = s == s ? s : -INFINITY;
    }
    __syncthreads();
    if (warp != 0) return;
    const bool live = !a.live || a.live[t];
    float biggest = -INFINITY;
    for (int e = lane; e < a.E; e += 32) biggest = fmaxf(biggest, logit[e]);
    for (int o = 16; o > 0; o >>= 1)
        biggest = fmaxf(biggest, __shfl_xor_sync(0xffffffffu, biggest, o));
    float sum = 0.0f;
    uint32_t taken = 0;  // bit i: expert lane + 32 i
    for (int e = lane; e < a.E; e += 32)
        sum += logit[e] == biggest ? 1.0f : expf(logit[e] - biggest);
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float chosen = 0.0f;
    for (int j = 0; j < a.top; ++j) {
        float best = -INFINITY;
        int at = kMoeMaxE;
        for (int i = 0; lane + 32 * i < a.E; ++i)
            if (!((taken >> i) & 1) && (logit[lane + 32 * i] > best || at == kMoeMaxE)) {
                best = logit[lane + 32 * i];
                at = lane + 32 * i;
            }
        for (int o = 16; o > 0; o >>= 1) {
            const float other = __shfl_xor_sync(0xffffffffu, best, o);
            const int other_at = __shfl_xor_sync(0xffffffffu, at, o);
            if (other_at < kMoeMaxE &&
                (at == kMoeMaxE || other > best || (other == best && other_at < at))) {
                best = other;
                at = other_at;
            }
        }
        if ((at & 31) == lane) taken |= 1u << (at >> 5);
        chosen += best == biggest ? 1.0f : expf(best - biggest);
    }
    // the chosen experts in ascending order
    int slot = 0;
    for (int i = 0; 32 * i < a.E; ++i) {
        const uint32_t mask = __ballot_sync(0xffffffffu, (taken >> i) & 1);
        if ((taken >> i) & 1) {
            const int e = lane + 32 * i;
            const int at = t * a.top + slot + __popc(mask & ((1u << lane) - 1));
            const float p = logit[e] == biggest ? 1.0f : expf(logit[e] - biggest);
            a.ids[at] = live ? e : -1;
            a.weights[at] = live ? p / (a.renormalize ? chosen : sum) : 0.0f;
        }
        slot += __popc(mask);
    }
}

// Adds column `col` of a tile times src[at .. at + N) (FP32 or 16-bit values).
__device__ float column_product(const uint8_t* tile, const Q4Geom& geom, int col, const void* src,
                                int dtype, size_t at) {
    float total = 0.0f;
    const int groups = kQ4UnitN / geom.group;
    for (int u = 0; u < geom.units; ++u) {
        const uint8_t* unit = tile + size_t(u) * geom.unit_bytes;
        for (int g = 0; g < groups; ++g) {
            float z = 8.0f;
            if (geom.zeros) z = unit[kQ4CodeBytes + groups * kQ4UnitK * 2 + g * kQ4UnitK + col];
            float acc = 0.0f;
            for (int i = g * geom.group / 8; i < (g + 1) * geom.group / 8; ++i) {
                const uint32_t w =
                    reinterpret_cast<const uint32_t*>(unit)[(i / 4 * kQ4UnitK + col) * 4 + i % 4];
                for (int e = 0; e < 8; ++e) {
                    const int n = u * kQ4UnitN + 8 * i + e;
                    if (n < geom.N)
                        acc = fmaf(float((w >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15) - z,
                                   load_as_float(src, dtype, at + n), acc);
                }
            }
            total = fmaf(q4_scale(reinterpret_cast<const uint16_t*>(unit + kQ4CodeBytes)[g * kQ4UnitK +
                                                                                        col],
                                  geom.fp16),
                         acc, total);
        }
    }
    return total;
}

__global__ void __launch_bounds__(kQ4UnitK)
    moe_hidden_kernel(MoeArgs a, const uint8_t* gate, const uint8_t* up, Q4Geom geom) {
    const int slot = blockIdx.y, t = slot / a.top, col = threadIdx.x;
    const int e = a.ids[slot], f = blockIdx.x * kQ4UnitK + col;
    if (e < 0 || f >= geom.K) return;
    const size_t at = e * geom.matrix_bytes() + blockIdx.x * geom.tile_bytes();
    const float g = column_product(gate + at, geom, col, a.x, a.dtype, t * a.ldx);
    const float u = column_product(up + at, geom, col, a.x, a.dtype, t * a.ldx);
    a.hidden[size_t(slot) * a.F + f] = g / (1.0f + expf(-g)) * u * a.weights[slot];
}

__global__ void __launch_bounds__(kQ4UnitK)
    moe_down_kernel(MoeArgs a, const uint8_t* down, Q4Geom geom) {
    const int t = blockIdx.y, col = threadIdx.x, d = blockIdx.x * kQ4UnitK + col;
    if (d >= geom.K) return;
    float v = 0.0f;
    for (int j = 0; j < a.top; ++j) {
        const int slot = t * a.top + j, e = a.ids[slot];
        if (e >= 0)
            v += column_product(down + e * geom.matrix_bytes() + blockIdx.x * geom.tile_bytes(), geom,
                                col, a.hidden, SGEMM_FLOAT32, size_t(slot) * a.F);
    }
    store_from_float(a.y, a.dtype, t * a.ldy + d, v);
}

bool stack_fits(const sgemm_q4& w, int E, int N, int K) {
    return q4_valid(&w) && w.data && aligned16(w.data) && w.count == E && w.N == N && w.K == K;
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" int sgemm_moe(const sgemm_moe_layer* layer, const void* x, long long ldx, int T,
                         const unsigned char* live, void* y, long long ldy, int* ids,
                         float* weights, void* stream) {
    if (!layer || !layer->router || !dtype_valid(layer->dtype) || !dtype_valid(layer->router_dtype))
        return SGEMM_ERR_ARG;
    const sgemm_moe_layer& m = *layer;
    if (m.D < 1 || m.D > kMoeMaxDim || m.F < 1 || m.F > kMoeMaxDim || m.E < 1 || m.E > kMoeMaxE ||
        m.top_k < 1 || m.top_k > kMoeMaxTop || m.top_k > m.E)
        return SGEMM_ERR_ARG;
    if (!stack_fits(m.gate, m.E, m.D, m.F) || !stack_fits(m.up, m.E, m.D, m.F) ||
        !stack_fits(m.down, m.E, m.F, m.D) || m.gate.group != m.up.group ||
        m.gate.flags != m.up.flags)
        return SGEMM_ERR_ARG;
    if (T < 0 || T > kMoeMaxT || ldx < m.D || ldy < m.D || ldx > (1ll << 40) || ldy > (1ll << 40))
        return SGEMM_ERR_ARG;
    if (T == 0) return SGEMM_OK;
    if (!x || !y) return SGEMM_ERR_ARG;
    const size_t size = dtype_bytes(m.dtype), side = size_t(T) * m.top_k * 4;
    const struct { const void* p; size_t bytes; } outs[3] = {
        {y, (size_t(T - 1) * ldy + m.D) * size}, {ids, ids ? side : 0}, {weights, weights ? side : 0}};
    const struct { const void* p; size_t bytes; } ins[6] = {
        {x, (size_t(T - 1) * ldx + m.D) * size},
        {m.router, size_t(m.E) * m.D * dtype_bytes(m.router_dtype)},
        {live, live ? size_t(T) : 0},
        {m.gate.data, q4_bytes(m.gate)}, {m.up.data, q4_bytes(m.up)}, {m.down.data, q4_bytes(m.down)}};
    for (int i = 0; i < 3; ++i) {
        if (!outs[i].bytes) continue;
        for (const auto& in : ins)
            if (in.bytes && ranges_overlap(outs[i].p, outs[i].bytes, in.p, in.bytes))
                return SGEMM_ERR_OVERLAP;
        for (int j = 0; j < i; ++j)
            if (outs[j].bytes && ranges_overlap(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes))
                return SGEMM_ERR_OVERLAP;
    }
    int dev = -1;
    if (!current_device(&dev)) return SGEMM_ERR_NO_DEVICE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const size_t slots = size_t(T) * m.top_k;
    Scratch ws;
    if (ws.alloc(dev, slots * 8 + slots * m.F * sizeof(float), s) != cudaSuccess)
        return SGEMM_ERR_CUDA;
    MoeArgs a;
    a.x = x;
    a.ldx = ldx;
    a.router = m.router;
    a.router_dtype = m.router_dtype;
    a.dtype = m.dtype;
    a.T = T;
    a.D = m.D;
    a.F = m.F;
    a.E = m.E;
    a.top = m.top_k;
    a.renormalize = m.renormalize;
    a.live = live;
    a.ids = ids ? ids : static_cast<int*>(ws.ptr);
    a.weights = weights ? weights : static_cast<float*>(ws.ptr) + slots;
    a.hidden = static_cast<float*>(ws.ptr) + 2 * slots;
    a.y = y;
    a.ldy = ldy;
    const Q4Geom g = q4_geom(m.gate), gd = q4_geom(m.down);
    moe_router_kernel<<<T, WARPS * 32, 0, s>>>(a);
    moe_hidden_kernel<<<dim3(g.tiles, int(slots)), kQ4UnitK, 0, s>>>(
        a, static_cast<const uint8_t*>(m.gate.data), static_cast<const uint8_t*>(m.up.data), g);
    moe_down_kernel<<<dim3(gd.tiles, T), kQ4UnitK, 0, s>>>(
        a, static_cast<const uint8_t*>(m.down.data), gd);
    count_launch(3);
    return cudaGetLastError() == cudaSuccess ? SGEMM_OK : SGEMM_ERR_CUDA;
}
