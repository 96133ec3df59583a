// moe_api.cu -- host side of the mixture-of-experts entry points of include/bsfp8.h:
// argument checks and launches of the router and of the layer for a few tokens.
#include <cuda_runtime.h>

#include <cstdint>

#include "bsfp8.h"
#include "host.h"
#include "moe_layer.cuh"
#include "moe_route.cuh"
#include "moe_tile.cuh"

namespace bsfp8 {

namespace {

template <int V>
void (*pick_kernel(int type))(RouteArgs) {
    return type == FP8_TYPE_BF16 ? bsfp8_route_pick<V, true> : bsfp8_route_pick<V, false>;
}

// A lane's experts: the least power of two that covers E.
int lane_experts(int E) {
    int v = 1;
    while (32 * v < E) v *= 2;
    return v;
}

void (*pick_kernel(int E, int type))(RouteArgs) {
    switch (lane_experts(E)) {
        case 1: return pick_kernel<1>(type);
        case 2: return pick_kernel<2>(type);
        case 4: return pick_kernel<4>(type);
        case 8: return pick_kernel<8>(type);
        case 16: return pick_kernel<16>(type);
        default: return pick_kernel<32>(type);
    }
}

bool set_shared(const void *kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

template <int MT>
bool set_down_shared() {
    return set_shared(reinterpret_cast<const void *>(bsfp8_moe_down<MT, 2>), moe_down_smem(MT)) &&
           set_shared(reinterpret_cast<const void *>(bsfp8_moe_down<MT, 8>), moe_down_smem(MT));
}

// The form for few tokens takes eight at a time: how often, and the pairs of eight tokens.
unsigned eights(int64_t T) { return static_cast<unsigned>((T + MOE_FEW_TOKENS - 1) / MOE_FEW_TOKENS); }
int64_t few_pairs(int64_t T, int64_t top) { return (T < MOE_FEW_TOKENS ? T : MOE_FEW_TOKENS) * top; }

template <int MT>
int launch_down(const MoeArgs &a, cudaStream_t stream) {
    return launch(few_pairs(a.T, a.top) <= 64 ? bsfp8_moe_down<MT, 2> : bsfp8_moe_down<MT, 8>,
                  dim3(static_cast<unsigned>((a.H + 16 * MT - 1) / (16 * MT)), 1, eights(a.T)), MOE_DOWN_WARPS * 32,
                  moe_down_smem(MT), 1, a, stream);
}

template <int NG>
bool set_tile_shared() {
    return set_shared(reinterpret_cast<const void *>(bsfp8_moe_tile<false, NG>), MT_SMEM) &&
           set_shared(reinterpret_cast<const void *>(bsfp8_moe_tile<true, NG>), MT_SMEM);
}

// The kernels of the layer for up to 8 NG tokens.
template <int NG>
int launch_tiles(MoeTileArgs &a, cudaStream_t stream) {
    int rc = encode_gate_up(&a.tmW, a.W1, a.E, a.I, a.H);
    if (rc != FP8_OK) return rc;
    a.ring = (MT_SMEM - smem_moe_fixed<false, NG>(a.T, a.top, a.E)) / 1024 * 1024;
    rc = launch(bsfp8_moe_tile<false, NG>, dim3(MT_CTAS), MT_THREADS, MT_SMEM, 1, a, stream);
    if (rc != FP8_OK) return rc;
    rc = encode_kmajor(&a.tmW, a.W2, static_cast<int64_t>(a.E) * a.H, a.I, MT_ROWS);
    if (rc != FP8_OK) return rc;
    a.ring = (MT_SMEM - smem_moe_fixed<true, NG>(a.T, a.top, a.E)) / 1024 * 1024;
    rc = launch(bsfp8_moe_tile<true, NG>, dim3(MT_CTAS), MT_THREADS, MT_SMEM, 1, a, stream);
    if (rc != FP8_OK) return rc;
    const dim3 grid(static_cast<unsigned>((a.H + MT_ROWS - 1) / MT_ROWS), static_cast<unsigned>(a.T));
    return launch(bsfp8_moe_join, grid, MT_JOIN_THREADS, 0, 1, a, stream);
}

// Tokens whose whole order one CTA makes.  8 of 64 experts in a graph, one CTA against two
// kernels: 32 tokens 5.3 us, 5.2; 64 tokens 7.7, 6.9; 128 tokens 12.3, 7.1.  The second launch
// costs a call of its own 1.3 us of the host's time.
constexpr int64_t kOneCtaTokens = 64;

// Tokens of a CTA of the ordered router: one CTA for few, else as even as the SMs allow.
int64_t route_chunk(int64_t T) {
    if (T <= kOneCtaTokens) return kOneCtaTokens;
    const int64_t even = (T + ROUTE_CHUNKS - 1) / ROUTE_CHUNKS;
    return even < ROUTE_WARPS ? ROUTE_WARPS : even;
}

int64_t route_chunks(int64_t T) { return T > 0 ? (T + route_chunk(T) - 1) / route_chunk(T) : 1; }

bool layer_sizes(int64_t T, int32_t top, int64_t I) {
    return T >= 0 && T <= FP8_MOE_MAX_TOKENS && top >= 1 && top <= FP8_MAX_TOP && I >= 0 && I < kLim && I % 16 == 0;
}

// The bytes of weights that T tokens read where routing is even.
double even_bytes(int64_t T, int32_t top, int32_t E, int64_t H, int64_t I) {
    double without = 1.0;   // an expert without tokens
    for (int64_t t = 0; t < T; ++t) without *= 1.0 - static_cast<double>(top < E ? top : E) / E;
    return (1.0 - without) * E * 3.0 * static_cast<double>(H) * static_cast<double>(I);
}

// Whether the tile form (moe_tile.cuh) serves the call, else the one for few tokens
// (moe_layer.cuh), whose set-up is 5 to 12 us shorter, whose rate falls as the tokens grow, and
// which reads an expert's weights again for each eight tokens (from L2).  By the weights that even
// routing reads; few-token form against tiles, us (hidden x inner), weights from HBM (and in L2, one
// call repeated):
//   4 to 8 tokens up from 120 MB: 5, 2 of 16 experts of 2048 x 1024 (49 MB) 18.1, 23.9 (15.1, 20.9); 8,
//     2 of 8 of 4096 x 1024 (91) 26.4, 31.8 (21.7, 27.3); 8, 7 of 7 of 6864 x 816 (118) 34.5, 42.1
//     (32.8, 39.3); 8, 4 of 32 of 2048 x 1024 (132) 38.4, 35.6; 8, 8 of 256 of 2048 x 512 (181) 48.7,
//     43.1; 8, 2 of 8 of 4096 x 14336 (1270) 225, 191; 8, 8 of 64 of 7168 x 2048 (1850) 289, 274
//   fewer from 400 MB: 1, 4 of 32 of 2048 x 1024 (25) 11.0, 21.8 (8.8, 20.8); 2, 8 of 64 of 4096 x 1536
//     (283) 60.8, 63.1; 1, 8 of 64 of 7168 x 2048 (352) 64.0, 66.0; 3, 1 of 8 of 4096 x 14336 (465)
//     98.8, 91.9; 2, 8 of 64 of 7168 x 2048 (660) 116.5, 115.4
//   more by what both cost with weights in L2 (HBM adds about as much to either): 6.5 us, 0.17 for each
//     MB that all eights read and 1.5 for 1000 CTAs of the up product, against 13.5, 0.8 for each token
//     of an expert and 0.09 for each MB.  4 of 24 of 768 x 256: 9 tokens 11.0, 16.7 (9.9, 15.2), 32 19.4,
//     20.2 (17.8, 18.8), 64 31.4, 25.2 (29.1, 24.6); 3 of 11 of 1344 x 512: 16 tokens 17.7, 21.0 (15.6,
//     19.7), 32 26.9, 24.1 (24.6, 22.7); 2 of 6 of 2048 x 1024: 9 tokens 18.6, 23.2 (16.6, 20.7), 24 29.2,
//     26.6 (25.2, 24.7); 8 of 32 of 1024 x 512: 9 tokens 26.5, 24.1 (24.1, 20.6); 2 of 16 of 2048 x 1024:
//     12 tokens 31.3, 27.7 (24.7, 22.0)
bool takes_tiles(int64_t T, int32_t top, int32_t E, int64_t H, int64_t I) {
    const double bytes = even_bytes(T, top, E, H, I);
    if (T <= MOE_FEW_TOKENS) return bytes >= (T < 4 ? 400e6 : 120e6);
    const double pairs = static_cast<double>(T) * top, ctas = pairs * static_cast<double>(I / MOE_UP_COLS);
    const double few = static_cast<double>(T / MOE_FEW_TOKENS) * even_bytes(MOE_FEW_TOKENS, top, E, H, I) +
                       even_bytes(T % MOE_FEW_TOKENS, top, E, H, I);
    return 6.5 + 0.17e-6 * few + 1.5e-3 * ctas > 13.5 + 0.8 * pairs / E + 0.09e-6 * bytes;
}

}  // namespace

int moe_setup() {
    for (int E = 32; E <= FP8_MAX_EXPERTS; E *= 2)
        for (int type : {FP8_TYPE_F32, FP8_TYPE_BF16})
            if (!set_shared(reinterpret_cast<const void *>(pick_kernel(E, type)), route_smem(E))) return FP8_ERR_CUDA;
    return set_shared(reinterpret_cast<const void *>(bsfp8_route_order), route_smem(FP8_MAX_EXPERTS)) &&
                   set_shared(reinterpret_cast<const void *>(bsfp8_moe_up<2>), MOE_UP_SMEM) &&
                   set_shared(reinterpret_cast<const void *>(bsfp8_moe_up<8>), MOE_UP_SMEM) && set_down_shared<1>() &&
                   set_down_shared<2>() && set_down_shared<3>() && set_tile_shared<1>() && set_tile_shared<2>() && set_tile_shared<4>() && set_tile_shared<8>()
               ? FP8_OK
               : FP8_ERR_CUDA;
}

}  // namespace bsfp8

using namespace bsfp8;

static_assert(MOE_MAX_TOKENS == FP8_MOE_MAX_TOKENS && MOE_MAX_TOP == FP8_MAX_TOP && ROUTE_MAX_TOP == FP8_MAX_TOP &&
                  MOE_MAX_EXPERTS == FP8_MAX_EXPERTS,
              "limits of the kernels and of the header");

extern "C" {

int64_t fp8_moe_route_workspace_bytes(int64_t T, int32_t E, int32_t top) {
    if (T < 0 || E < 1 || E > FP8_MAX_EXPERTS || top < 1 || top > FP8_MAX_TOP || top > E || T * top >= kLim) return 0;
    const int64_t chunks = route_chunks(T);
    return chunks > 1 ? int64_t(4) * E * chunks : 0;
}

int fp8_moe_route(const void *logits, int64_t ld, int type, int64_t T, int32_t E, int32_t top, int flags, float scale,
                  float *weights, int32_t *ids, int32_t *offsets, int32_t *rows, int32_t *places, void *workspace,
                  int64_t workspace_bytes, cudaStream_t stream) {
    if (type != FP8_TYPE_F32 && type != FP8_TYPE_BF16) return FP8_ERR_MODE;
    if (flags & ~(FP8_ROUTE_SIGMOID | FP8_ROUTE_ALL)) return FP8_ERR_MODE;
    if (T < 0 || T >= kLim || E < 1 || E > FP8_MAX_EXPERTS || top < 1 || top > FP8_MAX_TOP || top > E || ld < E ||
        ld >= 2 * kLim || T * top >= kLim)
        return FP8_ERR_SHAPE;
    const bool order = offsets != nullptr;
    if (!order && (rows || places)) return FP8_ERR_NULL;
    if (T == 0 && !order) return FP8_OK;
    if (T > 0 && (!logits || !weights || !ids || (order && (!rows || !places)))) return FP8_ERR_NULL;
    const int64_t need = order ? fp8_moe_route_workspace_bytes(T, E, top) : 0;
    if (need > 0 && !workspace) return FP8_ERR_NULL;
    if (need > 0 && workspace_bytes < need) return FP8_ERR_SHAPE;
    const int size = type == FP8_TYPE_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(weights, 4) || !aligned(ids, 4) || !aligned(offsets, 4) ||
        !aligned(rows, 4) || !aligned(places, 4) || (need > 0 && !aligned(workspace, 4)))
        return FP8_ERR_ALIGN;
    DeviceState *d = nullptr;
    int rc = device_setup(&d);
    if (rc != FP8_OK) return rc;
    RouteArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.weights = weights;
    a.ids = ids;
    a.offsets = offsets;
    a.rows = rows;
    a.places = places;
    a.counts = static_cast<int32_t *>(workspace);
    a.T = static_cast<int>(T);
    a.E = E;
    a.top = top;
    a.sigmoid = (flags & FP8_ROUTE_SIGMOID) != 0;
    a.all = (flags & FP8_ROUTE_ALL) != 0;
    a.scale = scale;
    // a lane loads its V neighbouring logits in pieces of up to 16 bytes, where every row
    // starts and ends at such a piece's boundary
    const int V = lane_experts(E), piece = V * size < 16 ? V * size : 16, values = piece / size;
    a.vec = E % values == 0 && ld % values == 0 && aligned(logits, piece);
    a.chunk = static_cast<int>(order ? route_chunk(T) : ROUTE_WARPS);
    a.chunks = static_cast<int>(order ? route_chunks(T) : (T + ROUTE_WARPS - 1) / ROUTE_WARPS);
    const int smem = order ? route_smem(E) : 0;
    rc = launch(pick_kernel(E, type), dim3(static_cast<unsigned>(a.chunks)), ROUTE_THREADS, smem, 1, a, stream);
    if (rc != FP8_OK || !order || a.chunks == 1) return rc;
    return launch(bsfp8_route_order, dim3(static_cast<unsigned>(a.chunks)), ROUTE_THREADS, smem, 1, a, stream);
}

int64_t fp8_moe_layer_workspace_bytes(int64_t T, int32_t top, int64_t I) {
    if (!layer_sizes(T, top, I)) return 0;
    return (T * top * (2 * I + I / 4) + 255) / 256 * 256 + int64_t(2) * MT_CTAS * T * MT_ROWS * 4 + 2 * MT_CTAS * 8 + 8;
}

int fp8_moe_layer(const void *x, const float *weights, const int32_t *ids, const void *W1, const float *s1,
                  const void *W2, const float *s2, void *out, int64_t T, int32_t top, int32_t E, int64_t H, int64_t I,
                  void *workspace, int64_t workspace_bytes, cudaStream_t stream) {
    if (!layer_sizes(T, top, I) || E < 0 || E > FP8_MAX_EXPERTS || H < 0 || H >= kLim || H % 16 != 0)
        return FP8_ERR_SHAPE;
    if (E * 2 * I >= 2 * kLim || E * H >= 2 * kLim) return FP8_ERR_SHAPE;
    if (T == 0 || H == 0) return FP8_OK;
    if (!out) return FP8_ERR_NULL;
    if (!aligned(out, 16)) return FP8_ERR_ALIGN;
    const bool work = E > 0 && I > 0;   // else the experts' sum is empty
    if (work) {
        if (!x || !weights || !ids || !W1 || !s1 || !W2 || !s2 || !workspace) return FP8_ERR_NULL;
        if (workspace_bytes < fp8_moe_layer_workspace_bytes(T, top, I)) return FP8_ERR_SHAPE;
        if (!aligned(x, 16) || !aligned(weights, 4) || !aligned(ids, 4) || !aligned(W1, 16) || !aligned(s1, 4) ||
            !aligned(W2, 16) || !aligned(s2, 4) || !aligned(workspace, 16))
            return FP8_ERR_ALIGN;
    }
    DeviceState *d = nullptr;
    int rc = device_setup(&d);
    if (rc != FP8_OK) return rc;
    if (!work) return zero_fill(out, T * H, stream);
    MoeTileArgs a{};
    a.x = static_cast<const __nv_bfloat16 *>(x);
    a.ids = ids;
    a.w = weights;
    a.W1 = static_cast<const uint8_t *>(W1);
    a.W2 = static_cast<const uint8_t *>(W2);
    a.s1 = s1;
    a.s2 = s2;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.h = static_cast<__half *>(workspace);
    a.hs = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + T * top * 2 * I);
    a.T = static_cast<int>(T);
    a.top = top;
    a.E = E;
    a.H = static_cast<int>(H);
    a.I = static_cast<int>(I);
    if (takes_tiles(T, top, E, H, I)) {
        uint8_t *rest = static_cast<uint8_t *>(workspace) + (T * top * (2 * I + I / 4) + 255) / 256 * 256;
        a.part = reinterpret_cast<float *>(rest);
        rest += int64_t(2) * MT_CTAS * T * MT_ROWS * 4;
        a.has = reinterpret_cast<unsigned long long *>(rest);
        a.busy = reinterpret_cast<int *>(rest + 2 * MT_CTAS * 8);
        a.status = d->status;
        a.wait_limit = wait_limit();
        a.withhold = withheld_stage();
        return guarded([&] {
            return T <= 8 ? launch_tiles<1>(a, stream) : T <= 16 ? launch_tiles<2>(a, stream) : T <= 32 ? launch_tiles<4>(a, stream) : launch_tiles<8>(a, stream);
        });
    }
    const MoeArgs &few = a;
    // words of pairs: two, or eight (8 tokens, 2 of 16 experts of 2048 x 1024: 17.8 us, 20.3)
    const int64_t pairs = few_pairs(T, top);
    const dim3 grid(static_cast<unsigned>(I / MOE_UP_COLS), static_cast<unsigned>(pairs), eights(T));
    rc = launch(pairs <= 64 ? bsfp8_moe_up<2> : bsfp8_moe_up<8>, grid, MOE_UP_WARPS * 32, MOE_UP_SMEM, 1, few, stream);
    if (rc != FP8_OK) return rc;
    // as many columns for a CTA as let one wave have all of them (one CTA on an SM), up to 48: 1
    // token, 8 of 64 experts of 7168 x 2048, 48 columns 63.6 us, 16 columns 73.5; 2 of 8 of 4096 x
    // 14336, 32 columns 70.2, 16 columns 76.9
    const int64_t wide = (H / 16 * eights(T) + d->sm_count - 1) / d->sm_count;
    return wide <= 1 ? launch_down<1>(few, stream) : wide == 2 ? launch_down<2>(few, stream) : launch_down<3>(few, stream);
}

}  // extern "C"
