// Host build of the rules of the token and int8 operators (token_launch.hpp), written
// out for the CPU tests as rows of int32.
//   token_rules_dump chunks OUT    n, cols, col, start, skip of every chunk of rows of n to 2100 columns
//   token_rules_dump form OUT CUS N K M...   the int8 product's form for M... rows of the experts, then how
//                                            many forms there are
//   token_rules_dump pieces OUT M...  m, each, pieces for the heights of the int8 product's tiles
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../../moe_grouped_block_mx_amd/csrc/token_launch.hpp"

int main(int argc, char** argv) {
  if (argc < 3) return 2;
  std::vector<int32_t> out;
  if (!std::strcmp(argv[1], "chunks")) {
    for (int n : {4, 8})
      for (int cols = n; cols <= 2100; ++cols)
        for (int col = 0; col < cols; col += n) {
          const mxgg::RowChunk c = mxgg::row_chunk(col, cols, n);
          for (int v : {n, cols, col, c.start, c.skip}) out.push_back(v);
        }
  } else if (!std::strcmp(argv[1], "form")) {
    mxgg::SplitArgs sp{};
    for (int a = 6; a < argc; ++a) sp.m[sp.G++] = (int)std::strtol(argv[a], nullptr, 10);
    out.push_back(mxgg::int8_form(sp, std::atoll(argv[4]), std::atoll(argv[5]), std::atoi(argv[3])));
    out.push_back(mxgg::kInt8Few44 + 1);
  } else if (!std::strcmp(argv[1], "pieces")) {
    for (int a = 3; a < argc; ++a)
      for (int each : {16, 32, 64, 128, 256}) {
        const int m = (int)std::strtol(argv[a], nullptr, 10);
        for (int v : {m, each, mxgg::token_pieces(m, each)}) out.push_back(v);
      }
  } else {
    return 2;
  }
  FILE* f = std::fopen(argv[2], "wb");
  if (!f) return 3;
  std::fwrite(out.data(), 4, out.size(), f);
  std::fclose(f);
  return 0;
}
