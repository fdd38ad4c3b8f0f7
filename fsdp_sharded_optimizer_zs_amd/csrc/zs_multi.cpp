// Entry points over many tensors (zs_multi_*, zs_adamw_multi, zs_grad_norm), of the
// 8-bit moments and of the 4-bit shards: host-side checks, then one launch. Nothing here
// allocates device memory or synchronizes.

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <vector>

#include "zs_multi.h"

#define ZS_EXPORT extern "C" __attribute__((visibility("default")))

using namespace zs;

// A checked table, as the chunks that the kernels take.
struct zs_multi {
    uint64_t magic;
    int32_t state;
    int32_t dtype;
    std::vector<MultiChunk> chunks;
    std::vector<Range> grads;    // what the gradients cover: sorted, disjoint
    std::vector<Range> written;  // what the step writes, likewise
};

namespace {

constexpr uint64_t kMagic = 0x7a736d756c746931ull;
constexpr int kBlock8 = 256;  // elements to a scale byte of the 8-bit moments
constexpr int kBlock4 = 32;   // elements to a scale byte of the 4-bit format

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0 ? 1 : 0); }

struct Owned {  // a range that the step writes, and whose it is
    Range r;
    int32_t tensor;
    const char* name;
};

zs_status check_multi(const char* who, const zs_multi* multi, const void* image) {
    if (multi == nullptr || multi->magic != kMagic)
        return fail(ZS_EINVAL, "%s: multi is NULL or not a live zs_multi", who);
    if (!multi->chunks.empty() && (image == nullptr || !aligned(image, 16)))
        return fail(ZS_EINVAL, "%s: image is NULL or not 16-byte aligned", who);
    return ZS_OK;
}

// The device image of a table: the kernels read it while they write.
Range image_range(const zs_multi& m, const void* image) {
    return range_of(image, int64_t(m.chunks.size() * sizeof(MultiChunk)), 1);
}

MultiImage image_of(const zs_multi& m, const void* image) {
    return MultiImage{static_cast<const MultiChunk*>(image), int64_t(m.chunks.size())};
}

// The chunks of one tensor, its arrays offset to each one's first element. The first chunk
// of a tensor that starts inside a cache line is shortened so that the others start where p
// (without a step: g) is at a multiple of 64 elements, and so are arrays laid out alike: a
// wavefront then covers whole lines. (1,000 ragged tensors end to end, 58M elements, fp32
// gradients and moments: 307 us against 377 with every chunk off the lines; the norm of
// 2,000: 130 against 131.) 8-bit moments cannot move off their blocks of 256.
void add_chunks(const zs_multi_tensor& x, int32_t t, int32_t state, int es,
                std::vector<MultiChunk>* out) {
    const int ms = state == ZS_STATE_F32 ? 4 : 1;
    const auto at = [](const void* base, int64_t bytes) -> void* {
        return base ? const_cast<char*>(static_cast<const char*>(base)) + bytes : nullptr;
    };
    int64_t end = ZS_MULTI_CHUNK;  // of the present chunk
    if (state != ZS_STATE_8BIT && x.numel > ZS_MULTI_CHUNK) {
        const uintptr_t place = state == ZS_STATE_F32 ? reinterpret_cast<uintptr_t>(x.p) / 4
                                                      : reinterpret_cast<uintptr_t>(x.g) / es;
        end -= int64_t(place % 64);
    }
    for (int64_t i = 0; i < x.numel; i = end, end += ZS_MULTI_CHUNK) {
        MultiChunk c{};
        if (state != ZS_STATE_NONE) {
            c.p = static_cast<float*>(at(x.p, i * 4));
            c.m = at(x.m, i * ms);
            c.v = at(x.v, i * ms);
            c.w_out = static_cast<uint16_t*>(at(x.w_out, i * 2));
        }
        if (state == ZS_STATE_8BIT) {
            c.m_scale = static_cast<uint8_t*>(at(x.m_scale, i / kBlock8));
            c.v_scale = static_cast<uint8_t*>(at(x.v_scale, i / kBlock8));
        }
        c.g = at(x.g, i * es);
        c.first = uint32_t(i);
        c.tensor = t;
        c.live = int32_t(std::min(x.numel, end) - i);
        out->push_back(c);
    }
}

zs_status check_max_norm(const char* who, double max_norm) {
    if (!(max_norm > 0.0)) return fail(ZS_EINVAL, "%s: max_norm must be > 0", who);
    return ZS_OK;
}

zs_status check_tensors(const zs_multi_tensor* ts, int32_t T, int32_t state, int es) {
    const char* who = "zs_multi_create";
    for (int32_t t = 0; t < T; ++t) {
        const zs_multi_tensor& x = ts[t];
        if (!size_ok(x.numel, 4))
            return fail(ZS_EINVAL, "%s: tensor %d has numel %lld", who, t, (long long)x.numel);
        if (x.numel == 0) continue;
        if (x.g == nullptr) return fail(ZS_EINVAL, "%s: tensor %d: g is NULL", who, t);
        if (!aligned(x.g, uintptr_t(es)))
            return fail(ZS_EINVAL, "%s: tensor %d: g not aligned to %d bytes", who, t, es);
        if (state == ZS_STATE_NONE) continue;
        if (!x.p || !x.m || !x.v)
            return fail(ZS_EINVAL, "%s: tensor %d: p, m or v is NULL", who, t);
        const bool f32 = state == ZS_STATE_F32;
        if (!aligned(x.p, 4) || (f32 && (!aligned(x.m, 4) || !aligned(x.v, 4))) ||
            !aligned(x.w_out, 2))
            return fail(ZS_EINVAL, "%s: tensor %d: p, m, v or w_out misaligned", who, t);
        if (f32 && (x.m_scale || x.v_scale))
            return fail(ZS_EINVAL, "%s: tensor %d: scales are for 8-bit moments only", who, t);
        if (!f32 && (!x.m_scale || !x.v_scale))
            return fail(ZS_EINVAL, "%s: tensor %d: m_scale or v_scale is NULL", who, t);
    }
    return ZS_OK;
}

// The ranges that the step writes, sorted.
std::vector<Owned> owned_ranges(const zs_multi_tensor* ts, int32_t T, int32_t state) {
    std::vector<Owned> own;
    if (state == ZS_STATE_NONE) return own;
    own.reserve(size_t(T) * 6);
    for (int32_t t = 0; t < T; ++t) {
        const zs_multi_tensor& x = ts[t];
        if (x.numel == 0) continue;
        const int ms = state == ZS_STATE_F32 ? 4 : 1;
        own.push_back({range_of(x.p, x.numel, 4), t, "p"});
        own.push_back({range_of(x.m, x.numel, ms), t, "m"});
        own.push_back({range_of(x.v, x.numel, ms), t, "v"});
        if (x.w_out) own.push_back({range_of(x.w_out, x.numel, 2), t, "w_out"});
        if (state == ZS_STATE_8BIT) {
            own.push_back({range_of(x.m_scale, ceil_div(x.numel, kBlock8), 1), t, "m_scale"});
            own.push_back({range_of(x.v_scale, ceil_div(x.numel, kBlock8), 1), t, "v_scale"});
        }
    }
    std::sort(own.begin(), own.end(),
              [](const Owned& a, const Owned& b) { return a.r.lo < b.r.lo; });
    return own;
}

// No written range may meet another one or a gradient. Two written ranges meet only if
// two neighbours do, and a gradient can only meet the last one that starts before its end.
zs_status check_alias(const zs_multi_tensor* ts, int32_t T, int es, const std::vector<Owned>& own) {
    const char* who = "zs_multi_create";
    for (size_t i = 1; i < own.size(); ++i)
        if (own[i - 1].r.hi > own[i].r.lo)
            return fail(ZS_EALIAS, "%s: %s of tensor %d overlaps %s of tensor %d", who, own[i].name,
                        own[i].tensor, own[i - 1].name, own[i - 1].tensor);
    for (int32_t t = 0; t < T; ++t) {
        if (ts[t].numel == 0) continue;
        const Range g = range_of(ts[t].g, ts[t].numel, es);
        auto it = std::lower_bound(own.begin(), own.end(), g.hi,
                                   [](const Owned& o, uintptr_t hi) { return o.r.lo < hi; });
        if (it != own.begin() && (it - 1)->r.hi > g.lo)
            return fail(ZS_EALIAS, "%s: g of tensor %d overlaps %s of tensor %d", who, t,
                        (it - 1)->name, (it - 1)->tensor);
    }
    return ZS_OK;
}

// The union of ranges: sorted, disjoint, those that touch joined.
std::vector<Range> merged(std::vector<Range> r) {
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
    size_t n = 0;
    for (size_t i = 0; i < r.size(); ++i) {
        if (n > 0 && r[i].lo <= r[n - 1].hi) r[n - 1].hi = std::max(r[n - 1].hi, r[i].hi);
        else r[n++] = r[i];
    }
    r.resize(n);
    return r;
}

// Whether x meets one of them.
bool meets(const std::vector<Range>& sorted, const Range& x) {
    auto it = std::lower_bound(sorted.begin(), sorted.end(), x.hi,
                               [](const Range& r, uintptr_t hi) { return r.lo < hi; });
    return it != sorted.begin() && (it - 1)->hi > x.lo;
}

// The checks that the moment conversions share.
zs_status check_state8(const char* who, int64_t S, int32_t kind) {
    if (kind != ZS_STATE8_M && kind != ZS_STATE8_V)
        return fail(ZS_EUNSUPPORTED, "%s: unknown kind %d", who, kind);
    if (!size_ok(S, 4)) return fail(ZS_EINVAL, "%s: S = %lld out of range", who, (long long)S);
    return ZS_OK;
}

}  // namespace

ZS_EXPORT zs_status zs_multi_create(const zs_multi_tensor* tensors, int32_t T, int32_t state,
                                    int32_t dtype, zs_multi** out) {
    const char* who = "zs_multi_create";
    if (out == nullptr) return fail(ZS_EINVAL, "%s: out is NULL", who);
    *out = nullptr;
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    if (state != ZS_STATE_NONE && state != ZS_STATE_F32 && state != ZS_STATE_8BIT)
        return fail(ZS_EUNSUPPORTED, "%s: unknown state %d", who, state);
    if (T < 0) return fail(ZS_EINVAL, "%s: T = %d < 0", who, T);
    if (T > 0 && tensors == nullptr) return fail(ZS_EINVAL, "%s: tensors is NULL", who);
    try {
        zs_status st = check_tensors(tensors, T, state, es);
        if (st != ZS_OK) return st;
        const std::vector<Owned> own = owned_ranges(tensors, T, state);
        st = check_alias(tensors, T, es, own);
        if (st != ZS_OK) return st;
        int64_t n = T;  // at most: a shortened first chunk can add one
        for (int32_t t = 0; t < T; ++t) n += ceil_div(tensors[t].numel, ZS_MULTI_CHUNK);
        std::unique_ptr<zs_multi> m(new zs_multi{kMagic, state, dtype, {}, {}, {}});
        std::vector<Range> g, w;
        for (int32_t t = 0; t < T; ++t)
            if (tensors[t].numel > 0) g.push_back(range_of(tensors[t].g, tensors[t].numel, es));
        for (const Owned& o : own) w.push_back(o.r);
        m->grads = merged(std::move(g));
        m->written = merged(std::move(w));
        m->chunks.reserve(size_t(n));
        for (int32_t t = 0; t < T; ++t) add_chunks(tensors[t], t, state, es, &m->chunks);
        *out = m.release();
    } catch (const std::exception&) {
        return fail(ZS_EINVAL, "%s: out of host memory", who);
    }
    return ok();
}

ZS_EXPORT zs_status zs_multi_image(const zs_multi* multi, const void** image, int64_t* bytes) {
    if (multi == nullptr || multi->magic != kMagic)
        return fail(ZS_EINVAL, "zs_multi_image: multi is NULL or not a live zs_multi");
    if (!image || !bytes) return fail(ZS_EINVAL, "zs_multi_image: an output pointer is NULL");
    *image = multi->chunks.data();
    *bytes = int64_t(multi->chunks.size() * sizeof(MultiChunk));
    return ok();
}

ZS_EXPORT zs_status zs_multi_destroy(zs_multi* multi) {
    if (multi == nullptr) return ok();
    if (multi->magic != kMagic)
        return fail(ZS_EINVAL, "zs_multi_destroy: not a live zs_multi");
    multi->magic = 0;
    delete multi;
    return ok();
}

ZS_EXPORT zs_status zs_adamw_multi(const zs_multi* multi, const void* image, const zs_adamw_hp* hp,
                                   const float* grad_scale, const zs_round_opts* round,
                                   hipStream_t stream) {
    const char* who = "zs_adamw_multi";
    zs_status st = check_multi(who, multi, image);
    if (st != ZS_OK) return st;
    if (multi->state == ZS_STATE_NONE)
        return fail(ZS_EINVAL, "%s: the table holds gradients only", who);
    st = check_hp(hp, who);
    if (st != ZS_OK) return st;
    if (!aligned(grad_scale, 4)) return fail(ZS_EINVAL, "%s: grad_scale not 4-byte aligned", who);
    if (grad_scale != nullptr && meets(multi->written, range_of(grad_scale, 1, 4)))
        return fail(ZS_EALIAS, "%s: grad_scale lies in an array that the step writes", who);
    if (!multi->chunks.empty() && meets(multi->written, image_range(*multi, image)))
        return fail(ZS_EALIAS, "%s: image overlaps an array that the step writes", who);
    MultiArgs a;
    bool stoch = false;
    a.rbc2s = 0.0f;
    a.seed_lo = a.seed_hi = 0;
    if (round != nullptr) {
        if (round->stochastic != 0 && round->stochastic != 1)
            return fail(ZS_EINVAL, "%s: stochastic must be 0 or 1", who);
        if (round->reserved != 0) return fail(ZS_EINVAL, "%s: reserved must be 0", who);
        stoch = round->stochastic == 1;
        a.seed_lo = uint32_t(round->seed);
        a.seed_hi = uint32_t(round->seed >> 32);
    }
    if (multi->chunks.empty()) return ok();
    a.k = adam_consts(*hp, 1);
    a.grad_scale = grad_scale;
    return hip_status(
        launch_multi(image_of(*multi, image), multi->state, multi->dtype, a, stoch, stream), who);
}

ZS_EXPORT zs_status zs_state8_layout(const int64_t* numels, int32_t T, int64_t* offsets_out) {
    const char* who = "zs_state8_layout";
    if (T < 0) return fail(ZS_EINVAL, "%s: T = %d < 0", who, T);
    if (T > 0 && numels == nullptr) return fail(ZS_EINVAL, "%s: numels is NULL", who);
    if (offsets_out == nullptr) return fail(ZS_EINVAL, "%s: offsets_out is NULL", who);
    int64_t at = 0;
    offsets_out[0] = 0;
    for (int32_t t = 0; t < T; ++t) {
        if (numels[t] < 0)
            return fail(ZS_EINVAL, "%s: numels[%d] = %lld < 0", who, t, (long long)numels[t]);
        if (numels[t] > INT64_MAX / 16 - at - 1024)
            return fail(ZS_EUNSUPPORTED, "%s: the buffer's size overflows", who);
        at += ceil_div(numels[t], 1024) * 1024;
        offsets_out[t + 1] = at;
    }
    return ok();
}

ZS_EXPORT zs_status zs_state8_encode(const float* x, int64_t S, int32_t kind, uint8_t* codes,
                                     uint8_t* scales, hipStream_t stream) {
    const char* who = "zs_state8_encode";
    zs_status st = check_state8(who, S, kind);
    if (st != ZS_OK) return st;
    if (S == 0) return ok();
    if (!x || !codes || !scales)
        return fail(ZS_EINVAL, "%s: x, codes or scales is NULL", who);
    if (!aligned(x, 4)) return fail(ZS_EINVAL, "%s: x not 4-byte aligned", who);
    const Range rx = range_of(x, S, 4), rc = range_of(codes, S, 1),
                rs = range_of(scales, ceil_div(S, kBlock8), 1);
    if (overlap(rx, rc) || overlap(rx, rs) || overlap(rc, rs))
        return fail(ZS_EALIAS, "%s: x, codes and scales overlap", who);
    return hip_status(launch_encode8(x, S, kind == ZS_STATE8_M, codes, scales, stream), who);
}

ZS_EXPORT zs_status zs_state8_decode(const uint8_t* codes, const uint8_t* scales, int64_t S,
                                     int32_t kind, int32_t dtype, void* out, hipStream_t stream) {
    const char* who = "zs_state8_decode";
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    zs_status st = check_state8(who, S, kind);
    if (st != ZS_OK) return st;
    if (S == 0) return ok();
    if (!out || !codes || !scales)
        return fail(ZS_EINVAL, "%s: codes, scales or out is NULL", who);
    if (!aligned(out, uintptr_t(es)))
        return fail(ZS_EINVAL, "%s: out not aligned to %d bytes", who, es);
    const Range ro = range_of(out, S, es);
    if (overlap(ro, range_of(codes, S, 1)) || overlap(ro, range_of(scales, ceil_div(S, kBlock8), 1)))
        return fail(ZS_EALIAS, "%s: out overlaps codes or scales", who);
    return hip_status(launch_decode8(codes, scales, S, kind == ZS_STATE8_M, dtype, out, stream),
                      who);
}

ZS_EXPORT zs_status zs_grad_norm(const zs_multi* multi, const void* image, double max_norm,
                                 double* sumsq, float* norm_coef, void* workspace,
                                 hipStream_t stream) {
    const char* who = "zs_grad_norm";
    zs_status st = check_multi(who, multi, image);
    if (st != ZS_OK) return st;
    st = check_max_norm(who, max_norm);
    if (st != ZS_OK) return st;
    if (!sumsq || !norm_coef || !workspace)
        return fail(ZS_EINVAL, "%s: sumsq, norm_coef or workspace is NULL", who);
    if (!aligned(sumsq, 8) || !aligned(norm_coef, 4) || !aligned(workspace, 16))
        return fail(ZS_EINVAL, "%s: sumsq, norm_coef or workspace misaligned", who);
    const Range out[3] = {range_of(sumsq, 1, 8), range_of(norm_coef, 2, 4),
                          range_of(workspace, ZS_NORM_WORKSPACE, 1)};
    for (int a = 0; a < 3; ++a)
        for (int b = a + 1; b < 3; ++b)
            if (overlap(out[a], out[b]))
                return fail(ZS_EALIAS, "%s: sumsq, norm_coef and workspace overlap", who);
    for (const Range& o : out)
        if (meets(multi->grads, o))
            return fail(ZS_EALIAS, "%s: an output or the workspace overlaps a gradient", who);
    for (const Range& o : out)
        if (overlap(image_range(*multi, image), o))
            return fail(ZS_EALIAS, "%s: an output or the workspace overlaps image", who);
    return hip_status(launch_norm(image_of(*multi, image), multi->dtype, max_norm, sumsq, norm_coef,
                                  static_cast<NormWorkspace*>(workspace), stream),
                      who);
}

ZS_EXPORT zs_status zs_clip_coef(const double* const* sumsq, int32_t D, double max_norm,
                                 float* norm_coef, hipStream_t stream) {
    const char* who = "zs_clip_coef";
    if (D < 1 || D > ZS_MAX_D) return fail(ZS_EINVAL, "%s: D = %d outside 1..%d", who, D, ZS_MAX_D);
    zs_status st = check_max_norm(who, max_norm);
    if (st != ZS_OK) return st;
    if (norm_coef == nullptr || !aligned(norm_coef, 4))
        return fail(ZS_EINVAL, "%s: norm_coef is NULL or misaligned", who);
    PtrPack sp;
    st = take_ptrs(reinterpret_cast<const void* const*>(sumsq), D, 8, "zs_clip_coef: sumsq", &sp);
    if (st != ZS_OK) return st;
    for (int r = 0; r < D; ++r)
        if (overlap(range_of(norm_coef, 2, 4), range_of(sp.p[r], 1, 8)))
            return fail(ZS_EALIAS, "%s: norm_coef overlaps sumsq[%d]", who, r);
    return hip_status(launch_clip(sp, D, max_norm, norm_coef, stream), who);
}

ZS_EXPORT zs_status zs_quantize_mx4(const void* src, int32_t dtype, int64_t S, uint8_t* codes,
                                    uint8_t* scales, hipStream_t stream) {
    const char* who = "zs_quantize_mx4";
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    if (!size_ok(S, 4)) return fail(ZS_EINVAL, "%s: S = %lld out of range", who, (long long)S);
    if (S == 0) return ok();
    if (!src || !codes || !scales) return fail(ZS_EINVAL, "%s: src, codes or scales is NULL", who);
    if (!aligned(src, uintptr_t(es)))
        return fail(ZS_EINVAL, "%s: src not aligned to %d bytes", who, es);
    const Range rx = range_of(src, S, es), rc = range_of(codes, ceil_div(S, 2), 1),
                rs = range_of(scales, ceil_div(S, kBlock4), 1);
    if (overlap(rx, rc) || overlap(rx, rs) || overlap(rc, rs))
        return fail(ZS_EALIAS, "%s: src, codes and scales overlap", who);
    return hip_status(launch_quantize_mx4(src, dtype, S, codes, scales, stream), who);
}

ZS_EXPORT zs_status zs_gather_unit_mx4(const uint8_t* const* codes, const uint8_t* const* scales,
                                       int32_t D, int64_t S, int32_t dtype, void* flat_out,
                                       hipStream_t stream) {
    const char* who = "zs_gather_unit_mx4";
    const int es = elem_size(dtype);
    if (es == 0) return fail(ZS_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
    if (D < 1 || D > ZS_MAX_D) return fail(ZS_EINVAL, "%s: D = %d outside 1..%d", who, D, ZS_MAX_D);
    if (!size_ok(S, es) || S > INT64_MAX / 16 / es / D)
        return fail(ZS_EINVAL, "%s: S = %lld out of range", who, (long long)S);
    if (S == 0) return ok();
    if (flat_out == nullptr || !aligned(flat_out, uintptr_t(es)))
        return fail(ZS_EINVAL, "%s: flat_out is NULL or not aligned to %d bytes", who, es);
    PtrPack cp, sp;
    zs_status st = take_ptrs(reinterpret_cast<const void* const*>(codes), D, 1,
                             "zs_gather_unit_mx4: codes", &cp);
    if (st != ZS_OK) return st;
    st = take_ptrs(reinterpret_cast<const void* const*>(scales), D, 1,
                   "zs_gather_unit_mx4: scales", &sp);
    if (st != ZS_OK) return st;
    const Range out = range_of(flat_out, S * D, es);
    for (int r = 0; r < D; ++r)
        if (overlap(out, range_of(cp.p[r], ceil_div(S, 2), 1)) ||
            overlap(out, range_of(sp.p[r], ceil_div(S, kBlock4), 1)))
            return fail(ZS_EALIAS, "%s: flat_out overlaps codes or scales of shard %d", who, r);
    return hip_status(launch_gather_mx4(cp, sp, D, S, dtype, flat_out, stream), who);
}
