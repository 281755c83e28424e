// Host build of the few-token expert layer's plan (how a call is cut, its LDS and
// workspace) over every number of tokens and choices, written out for the CPU
// tests: per call one row of int32.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "../../moe_grouped_block_mx_amd/csrc/block_launch.hpp"

int main(int argc, char** argv) {
  if (argc != 2) return 2;
  std::vector<int32_t> experts, out;
  for (int e = 1; e <= 512; e += e < 24 ? 1 : e < 128 ? 8 : 24) experts.push_back(e);
  experts.push_back(512);
  for (int fmt = 0; fmt < 3; ++fmt)
    for (int hidden : {32, 1056, 4096, 6144, 65536})
      for (int tokens = 1; tokens <= mxgg::kMoeTokens; ++tokens)
        for (int top_k = 1; top_k <= mxgg::kMoeTopK; ++top_k)
          for (int e : experts) {
            if (top_k > e) continue;
            mxgg::MoeParams p{};
            p.tokens = tokens;
            p.top_k = top_k;
            p.experts = e;
            p.hidden = hidden;
            p.inner = 32;
            p.rows = tokens * top_k;
            mxgg::moe_plan(p, (mxgg::MoeFormat)fmt);
            const mxgg::MoeWorkspace w = mxgg::moe_workspace(tokens, e, top_k, p.inner);
            for (int64_t v : {(int64_t)fmt, (int64_t)hidden, (int64_t)tokens, (int64_t)top_k, (int64_t)e, (int64_t)p.segment,
                              (int64_t)p.dmas, (int64_t)p.most_segments, (int64_t)p.down_tiles, (int64_t)p.splits,
                              (int64_t)mxgg::moe_up_lds(p), (int64_t)mxgg::moe_down_lds(p),
                              (int64_t)((w.rows - w.segments) / sizeof(mxgg::MoeSegment)),
                              (int64_t)((w.inner - w.parts) / 4)})
              out.push_back((int32_t)v);
          }
  FILE* f = std::fopen(argv[1], "wb");
  if (!f) return 3;
  std::fwrite(out.data(), 4, out.size(), f);
  std::fclose(f);
  return 0;
}
