// Exercises the host side of the entry points of the rest of a layer (argument checks,
// workspace sizing, empty problems) for a build whose host code runs under
// AddressSanitizer and UndefinedBehaviorSanitizer.  Every call returns before any
// device work.  Exit status 0 on success, 1 on an unexpected result.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include "naju.h"

static int failures = 0;

static void expect(const char *what, naju_status_t got, naju_status_t want)
{
    const char *msg = naju_last_error();
    if (got != want || (got != NAJU_OK && std::strlen(msg) == 0)) {
        std::fprintf(stderr, "%s: status %d, expected %d (%s)\n", what, (int)got, (int)want, msg);
        ++failures;
    }
}

static void refused(const char *what, naju_status_t got)
{
    if (got == NAJU_OK) {
        std::fprintf(stderr, "%s: accepted\n", what);
        ++failures;
    }
}

int main()
{
    alignas(256) static unsigned char buf[1 << 12];
    void *p = buf, *mis = buf + 1;
    float *fp = (float *)buf;
    const size_t big = (size_t)1 << 60;

    const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 8, 63, 64, 65, 4096, 8192, 8193, (int64_t)1 << 20,
                             ((int64_t)1 << 20) + 1, (int64_t)1 << 30, (int64_t)1 << 40,
                             ((int64_t)1 << 40) + 1, INT64_MAX};
    for (int64_t T : sizes)
        for (int64_t d : sizes) {
            (void)naju_res_norm_bwd_workspace_bytes(T, d);
            const naju_status_t s =
                naju_res_norm_fwd(T, d, NAJU_BF16, NAJU_F32, nullptr, nullptr, nullptr, nullptr,
                                  nullptr, fp, 1e-6f, nullptr, p, nullptr);
            if (T != 0 && d != 0) refused("res_norm_fwd without x", s);
            const naju_status_t b = naju_res_norm_bwd(
                T, d, NAJU_F32, NAJU_F32, NAJU_F32, nullptr, nullptr, nullptr, nullptr, nullptr,
                nullptr, nullptr, nullptr, 0.f, nullptr, nullptr, nullptr, nullptr, nullptr,
                nullptr, nullptr, 0, nullptr);
            if (T != 0 && d != 0) refused("res_norm_bwd without gradients", b);
        }
    expect("res_norm_bwd workspace",
           naju_res_norm_bwd(8, 64, NAJU_F32, NAJU_F32, NAJU_F32, p, nullptr, p, nullptr, nullptr,
                             nullptr, nullptr, fp, 1e-6f, p, nullptr, nullptr, nullptr, nullptr,
                             fp, p, 16, nullptr),
           NAJU_EWORKSPACE);
    expect("res_norm_fwd alignment",
           naju_res_norm_fwd(8, 64, NAJU_BF16, NAJU_F32, mis, nullptr, nullptr, nullptr, nullptr,
                             fp, 1e-6f, nullptr, p, nullptr),
           NAJU_EINVAL);

    const int64_t counts[] = {INT64_MIN, -1, 0, 1, 3, 8, 200, 65535, 65536, (int64_t)1 << 20,
                              (int64_t)1 << 30, ((int64_t)1 << 30) + 1, INT64_MAX};
    const int64_t dims[] = {-8, 0, 1, 8, 12, 128, 256, 264, INT64_MAX};
    for (int64_t B : counts)
        for (int64_t L : counts)
            for (int64_t H : counts)
                for (int64_t Hk : {(int64_t)0, (int64_t)1, (int64_t)3, H})
                    for (int64_t d : dims) {
                        const size_t f = naju_linattn_fwd_workspace_bytes(B, L, H, Hk, d, 8);
                        const size_t b = naju_linattn_bwd_workspace_bytes(B, L, H, Hk, 16, d);
                        if (f > big || b > big) {
                            std::fprintf(stderr, "workspace sizes wrapped\n");
                            ++failures;
                        }
                        const naju_status_t s = naju_linattn_fwd(
                            B, L, H, Hk, d, 8, NAJU_BF16, nullptr, 4096, nullptr, 4096, nullptr,
                            4096, fp, nullptr, nullptr, 1.f, nullptr, nullptr, nullptr, 0,
                            nullptr);
                        if (B > 0 && L > 0 && H > 0) refused("linattn_fwd without q", s);
                        if (B > 0 && H > 0)
                            refused("linattn_step without q",
                                    naju_linattn_step(B, H, Hk, d, 8, NAJU_F32, nullptr, nullptr,
                                                      nullptr, fp, fp, 1.f, nullptr, fp, nullptr));
                    }
    expect("linattn_fwd workspace",
           naju_linattn_fwd(1, 65536, 2, 2, 64, 64, NAJU_BF16, p, 128, p, 128, p, 128, fp, nullptr,
                            nullptr, 1.f, p, nullptr, p, 16, nullptr),
           NAJU_EWORKSPACE);
    expect("linattn_bwd stride",
           naju_linattn_bwd(1, 8, 2, 1, 64, 64, NAJU_BF16, p, 128, p, 63, p, 64, fp, nullptr,
                            nullptr, 1.f, p, nullptr, p, p, p, nullptr, p, big, nullptr),
           NAJU_EINVAL);

    // lists of tensors: sizes, gaps, overlaps, repeats
    for (int64_t n : {(int64_t)-1, (int64_t)0, (int64_t)1, ((int64_t)1 << 24) + 1, INT64_MAX})
        if (n != 0)
            refused("adamw_step without tensors",
                    naju_adamw_step(n, nullptr, NAJU_F32, 32, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1,
                                    nullptr, nullptr, nullptr, nullptr));
    std::vector<naju_adamw_tensor_t> list(1000);
    for (size_t i = 0; i < list.size(); ++i) {
        naju_adamw_tensor_t t{};
        t.n = (int64_t)(i * 7919 % 37);
        t.p = fp + 4096 * ((i * 389) % list.size());
        t.g = t.m = t.v = buf;
        t.m_scale = t.v_scale = fp;
        list[i] = t;
    }
    auto step = [&](int bits, int64_t at) {
        return naju_adamw_step((int64_t)list.size(), list.data(), NAJU_BF16, bits, 1e-3, 0.9,
                               0.999, 1e-8, 0.0, at, nullptr, nullptr, nullptr, nullptr);
    };
    expect("adamw_step number", step(8, 0), NAJU_EINVAL);
    expect("adamw_step bits", step(16, 1), NAJU_EUNSUPPORTED);
    const naju_adamw_tensor_t kept = list[500];
    list[500].n = 5;
    list[500].p = list[501].p;
    list[501].n = 1;
    expect("adamw_step repeats", step(32, 1), NAJU_EINVAL);
    list[500] = kept;
    list[700].n = INT64_MAX;
    expect("adamw_step size", step(32, 1), NAJU_EINVAL);
    list[700].n = 3;
    list[700].m = nullptr;
    expect("adamw_step states", step(32, 1), NAJU_EINVAL);
    for (auto &t : list) t.n = 0;
    expect("adamw_step of nothing", step(32, INT64_MAX), NAJU_OK);

    if (failures == 0) std::printf("layer driver: ok\n");
    return failures == 0 ? 0 : 1;
}
