// The plan of items of single-token attention, on the host: "R n0 n1 ..." a line (tiles of each sequence, nxN for N
// equal ones) in; for the least and the safe chunk: "chunk items slots splits" out.
#include <cstdio>
#include <iostream>
#include <sstream>
#include <string>
#include <vector>

#include "../flash_attention_backward_gb300/csrc/fa_decode.cuh"

int main() {
  std::string line;
  while (std::getline(std::cin, line)) {
    std::istringstream in(line);
    int R;
    in >> R;
    std::vector<long long> n, times;
    long long U = 0, B = 0;
    for (std::string w; in >> w;) {
      const size_t x = w.find('x');
      n.push_back(std::stoll(w)), times.push_back(x == std::string::npos ? 1 : std::stoll(w.substr(x + 1)));
      U += n.back() * times.back(), B += times.back();
    }
    for (int safe = 0; safe < 2; ++safe) {
      const int chunk = safe ? fap::safe_chunk(U, (int)B, R) : fap::least_chunk(U, R);
      long long items = 0, slots = 0, split = 0;
      for (size_t i = 0; i < n.size(); ++i) {
        const fap::Counts c = fap::unpack_counts(fap::pack_counts((int)n[i], chunk));
        items += c.items * times[i], slots += c.slots * times[i], split += c.split * times[i];
      }
      std::printf("%d %lld %lld %lld%c", chunk, items, slots, split, safe ? '\n' : ' ');
    }
  }
}
